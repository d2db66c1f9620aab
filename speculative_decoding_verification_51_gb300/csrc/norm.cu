// norm.cu -- the norm of each head of queries and keys with the rotation in the same
// pass (rotate.cuh): to tensors (spec_norm_rope), or on the way into the cache
// (spec_norm_kv_write), where the keys can go to a tensor as well.
//
//   y = x / sqrt(mean(x^2) + eps) * w over the head's channels, then the rotation
//
// in float32 with one rounding at the end.  The lanes that hold a head's channels add
// up their squares and join the sums by shuffles; weights and angles are one factor each,
// made when a lane turns to another tensor.  Bound by instructions and HBM: 32771 tokens of 40
// heads of 128 channels take 114 us (0.87 of the measured copy rate) at two CTAs an SM; 4608
// tokens into an 8-bit cache and back 36.
#include "rotate.cuh"

using namespace sv;

namespace {

spec_status check_norm(const spec_head_norm* n) {
    if (n->dtype != SPEC_F32 && n->dtype != SPEC_BF16 && n->dtype != SPEC_F16) return SPEC_ERR_INVALID_ARG;
    if (!(n->eps >= 0.f) || !(n->eps < 3.4e38f)) return SPEC_ERR_INVALID_ARG;
    const size_t es = dtype_bytes(n->dtype);
    return aligned(n->q_weight, es) && aligned(n->k_weight, es) ? SPEC_OK : SPEC_ERR_UNSUPPORTED;
}

void put_norm(RotArgs& A, const spec_head_norm* n) {
    A.eps = n ? n->eps : -1.f;
    A.w[0] = n ? n->q_weight : nullptr;
    A.w[1] = n ? n->k_weight : nullptr;
    A.w_dtype = n ? n->dtype : SPEC_F32;
}

void put_table(RotArgs& A, const spec_rope_table* t, const int32_t* positions) {
    if (!t) return;
    A.pos = positions;
    A.turns = reinterpret_cast<const unsigned long long*>(t->turns);
    A.half_rot = t->rot / 2;
    A.interleaved = t->layout == SPEC_ROPE_INTERLEAVED;
    A.scale = t->scale;
}

}  // namespace

extern "C" {

spec_status spec_norm_rope(const spec_head_norm* norm, const void* q, int q_heads, int64_t q_token_stride,
                           int64_t q_head_stride, void* out_q, int64_t oq_token_stride,
                           int64_t oq_head_stride, const void* k, int k_heads, int64_t k_token_stride,
                           int64_t k_head_stride, void* out_k, int64_t ok_token_stride,
                           int64_t ok_head_stride, spec_dtype dtype, int D, int64_t T,
                           const int32_t* positions, const spec_rope_table* table, spec_stream_t stream) {
    if (T < 0 || q_heads < 0 || k_heads < 0 || q_heads > 65536 || k_heads > 65536 || D < 2 ||
        T > (1ll << 40) || !norm)
        return SPEC_ERR_INVALID_ARG;
    if (dtype != SPEC_F32 && dtype != SPEC_BF16 && dtype != SPEC_F16) return SPEC_ERR_INVALID_ARG;
    if (D > MAX_ROW || D % 2) return SPEC_ERR_UNSUPPORTED;
    const spec_status ns = check_norm(norm);
    if (ns != SPEC_OK) return ns;
    if (table) {
        const spec_status ts = check_table(table, D);
        if (ts != SPEC_OK) return ts;
    }
    if (T == 0 || q_heads + k_heads == 0) return SPEC_OK;
    if ((table && !positions) || (q_heads && (!q || !out_q)) || (k_heads && (!k || !out_k)))
        return SPEC_ERR_INVALID_ARG;
    const size_t es = dtype_bytes(dtype);
    if (!aligned(q, es) || !aligned(k, es) || !aligned(out_q, es) || !aligned(out_k, es) || !aligned(positions, 4))
        return SPEC_ERR_UNSUPPORTED;
    RotArgs A = {};
    A.q = {q, out_q, q_token_stride, q_head_stride, oq_token_stride, oq_head_stride, q_heads};
    A.k = {k, out_k, k_token_stride, k_head_stride, ok_token_stride, ok_head_stride, k_heads};
    put_table(A, table, positions);
    put_norm(A, norm);
    A.sign = 1.f;
    A.D = D;
    A.T = T;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == SPEC_F32    ? launch_rotate_vec<float, false, NORM>(A, st)
                          : dtype == SPEC_BF16 ? launch_rotate_vec<__nv_bfloat16, false, NORM>(A, st)
                                               : launch_rotate_vec<__half, false, NORM>(A, st);
    return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

spec_status spec_norm_kv_write(const spec_kv_cache* cache, const spec_head_norm* norm, const void* k,
                               int64_t k_token_stride, int64_t k_head_stride, void* out_k,
                               int64_t ok_token_stride, int64_t ok_head_stride, const void* v,
                               int64_t v_token_stride, int64_t v_head_stride, spec_dtype dtype, int64_t T,
                               const int64_t* slots, const int32_t* positions, const spec_rope_table* table,
                               const void* q, int q_heads, int64_t q_token_stride, int64_t q_head_stride,
                               void* out_q, int64_t oq_token_stride, int64_t oq_head_stride,
                               int32_t* dev_status, spec_stream_t stream) {
    const spec_status cs = check_cache(cache);
    if (cs != SPEC_OK) return cs;
    if (T < 0 || T > (1ll << 40) || q_heads < 0 || q_heads > 65536) return SPEC_ERR_INVALID_ARG;
    const bool e4 = cache->dtype == SPEC_E4M3;
    if (dtype != SPEC_F32 && dtype != SPEC_BF16 && dtype != SPEC_F16) return SPEC_ERR_INVALID_ARG;
    if (!e4 && int(dtype) != cache->dtype) return SPEC_ERR_INVALID_ARG;
    if (norm) {
        const spec_status ns = check_norm(norm);
        if (ns != SPEC_OK) return ns;
    }
    if (table) {
        const spec_status ts = check_table(table, cache->head_dim);
        if (ts != SPEC_OK) return ts;
        if (!positions && T > 0) return SPEC_ERR_INVALID_ARG;
    }
    if (q_heads && !table && !norm) return SPEC_ERR_INVALID_ARG;  // queries come along to be changed
    if (T == 0) return SPEC_OK;
    if (!k || !v || !slots || (q_heads && (!q || !out_q))) return SPEC_ERR_INVALID_ARG;
    const size_t es = dtype_bytes(dtype);
    if (!aligned(k, es) || !aligned(v, es) || !aligned(q, es) || !aligned(out_q, es) || !aligned(out_k, es) ||
        !aligned(slots, 8) || !aligned(positions, 4) || !aligned(dev_status, 4))
        return SPEC_ERR_UNSUPPORTED;
    RotArgs A = {};
    if (q_heads)
        A.q = {q, out_q, q_token_stride, q_head_stride, oq_token_stride, oq_head_stride, q_heads};
    A.k = {k, out_k, k_token_stride, k_head_stride, ok_token_stride, ok_head_stride, cache->heads};
    A.v = {v, nullptr, v_token_stride, v_head_stride, 0, 0, cache->heads};
    put_table(A, table, positions);
    put_norm(A, norm);
    A.sign = 1.f;
    A.D = cache->head_dim;
    A.T = T;
    A.c = view_of(*cache);
    A.slots = reinterpret_cast<const long long*>(slots);
    A.status = dev_status;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = e4                   ? launch_norm_e4m3(A, dtype, st)
                          : dtype == SPEC_BF16 ? launch_rotate_vec<__nv_bfloat16, false, NORM>(A, st)
                                               : launch_rotate_vec<__half, false, NORM>(A, st);
    return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"
