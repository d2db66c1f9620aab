// tree_attn_e4m3.cu -- k_attn_rows over a cache of type e4m3.
#include "tree_attn_rows.cuh"

namespace sv {
cudaError_t launch_attn_e4m3(const AttnLaunch& L, int mt) { return launch_rows_any<SPEC_E4M3>(L, mt); }
}  // namespace sv
