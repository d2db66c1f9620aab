// tree_attn_bf16.cu -- the attention kernels over a cache of type bf16.
#include "tree_attn_rows.cuh"
#include "tree_attn_tiles.cuh"

namespace sv {
cudaError_t launch_attn_bf16(const AttnLaunch& L, bool tiles) {
    if (tiles) return L.A.D <= 64 ? launch_tiles<SPEC_BF16, 64>(L) : launch_tiles<SPEC_BF16, 128>(L);
    return launch_rows_any<SPEC_BF16>(L);
}
}  // namespace sv
