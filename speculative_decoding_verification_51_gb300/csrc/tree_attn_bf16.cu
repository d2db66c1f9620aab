// tree_attn_bf16.cu -- k_attn_rows over a cache of type bf16.
#include "tree_attn_rows.cuh"

namespace sv {
cudaError_t launch_attn_bf16(const AttnLaunch& L, int mt) { return launch_rows_any<SPEC_BF16>(L, mt); }
}  // namespace sv
