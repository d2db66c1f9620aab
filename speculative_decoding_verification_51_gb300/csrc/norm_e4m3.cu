// norm_e4m3.cu -- norms and rotation on the way into an 8-bit cache (norm.cu).
#include "rotate.cuh"

namespace sv {
cudaError_t launch_norm_e4m3(const RotArgs& A, int dtype, cudaStream_t st) {
    return dtype == SPEC_F32    ? launch_rotate_vec<float, true, NORM>(A, st)
           : dtype == SPEC_BF16 ? launch_rotate_vec<__nv_bfloat16, true, NORM>(A, st)
                                : launch_rotate_vec<__half, true, NORM>(A, st);
}
}  // namespace sv
