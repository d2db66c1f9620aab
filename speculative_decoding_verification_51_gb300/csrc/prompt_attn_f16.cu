// prompt_attn_f16.cu -- attention over whole prompts of type f16.
#include "prompt_attn.cuh"

namespace sv {
cudaError_t launch_prompt_f16(const PromptLaunch& L) { return launch_prompt_any<true>(L); }
}  // namespace sv
