// tree_attn_f16.cu -- k_attn_rows over a cache of type f16.
#include "tree_attn_rows.cuh"

namespace sv {
cudaError_t launch_attn_f16(const AttnLaunch& L, int mt) { return launch_rows_any<SPEC_F16>(L, mt); }
}  // namespace sv
