// prompt_attn_bf16.cu -- attention over whole prompts of type bf16.
#include "prompt_attn.cuh"

namespace sv {
cudaError_t launch_prompt_bf16(const PromptLaunch& L) { return launch_prompt_any<false>(L); }
}  // namespace sv
