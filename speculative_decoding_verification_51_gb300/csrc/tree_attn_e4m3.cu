// tree_attn_e4m3.cu -- the attention kernels over a cache of type e4m3.
#include "tree_attn_rows.cuh"
#include "tree_attn_tiles_e4m3.cuh"

namespace sv {
cudaError_t launch_attn_e4m3(const AttnLaunch& L, bool tiles) {
    if (tiles) return L.A.D <= 64 ? launch_tiles_e4m3<64>(L) : launch_tiles_e4m3<128>(L);
    return launch_rows_any<SPEC_E4M3>(L);
}
}  // namespace sv
