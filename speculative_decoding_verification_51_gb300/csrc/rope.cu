// rope.cu -- rotary positions, and the cache rows written and read.
//
// The heads of a token are turned by its position's angles and stored: to a
// tensor (spec_rope), or to the token's cache slot, as they are or in 8 bits
// (spec_kv_write).
//
// The kernels that turn are in rotate.cuh.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "rotate.cuh"

namespace sv {

int sm_count() {
    static std::mutex mu;
    static int sms[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lk(mu);
    if (!sms[dev] && cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return sms[dev];
}

namespace {

// Rows of T slots: one thread per 16 bytes of a (token, head)'s row as it is
// written, so that a warp's stores leave no gaps.  I: the type
// of the indexes (32 bits where they are enough: a division of 64 costs more than
// the copy).
template <typename C, typename T, typename I>
__global__ void __launch_bounds__(256) k_kv_read(const __grid_constant__ CacheView c, long long T_,
                                                 const long long* slots, T* out_k, T* out_v) {
    begin_after_previous();
    constexpr int VEC = 16 / sizeof(T);
    const I vecs = c.D / VEC, heads = c.heads, n = I(T_) * heads * vecs;
    for (I i = blockIdx.x * I(256) + threadIdx.x; i < n; i += gridDim.x * I(256)) {
        const I th = i / vecs, t = th / heads;
        const int d = int(i - th * vecs) * VEC, h = int(th - t * heads);
        const long long slot = slots[t];
        Words<C, VEC> k, v;
        float fk = 1.f, fv = 1.f;
#pragma unroll
        for (int e = 0; e < VEC * int(sizeof(C)) / 4; ++e) k.w[e] = v.w[e] = 0;
        if (slot >= 0 && slot < c.slots) {
            const long long p = sizeof(I) == 4 ? (long long)(uint32_t(slot) / uint32_t(c.page)) : slot / c.page;
            const int o = int(slot - p * c.page);
            const long long at = p * c.page_stride + h * c.head_stride + o * c.token_stride + d;
            k = *reinterpret_cast<const Words<C, VEC>*>(static_cast<const C*>(c.k) + at);
            v = *reinterpret_cast<const Words<C, VEC>*>(static_cast<const C*>(c.v) + at);
            if constexpr (sizeof(C) == 1) {
                const long long sr = (p * c.heads + h) * c.page + o;
                fk = exp2_int(min(max(int(c.ks[sr]), 1), 253) - 127);
                fv = exp2_int(min(max(int(c.vs[sr]), 1), 253) - 127);
            }
        }
        auto write = [&](const Words<C, VEC>& x, float f, T* out) {
            Words<T, VEC> w;
#pragma unroll
            for (int e = 0; e < VEC / 2; ++e) {
                float2 a;
                if constexpr (sizeof(C) == 1) {
                    const uint32_t b = e4m3x2_to_f16x2(uint16_t(x.w[e / 2] >> (16 * (e & 1))));
                    a = __half22float2(*reinterpret_cast<const __half2*>(&b));
                    a.x *= f;
                    a.y *= f;
                } else {
                    a = get2(x, e);
                }
                set2(w, e, a.x, a.y);
            }
            *reinterpret_cast<Words<T, VEC>*>(out + (long long)i * VEC) = w;
        };
        write(k, fk, out_k);
        write(v, fv, out_v);
    }
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

spec_status spec_rope_turns(int rot, double base, int scaling, double factor, double original_len,
                            double fast, double slow, uint64_t* out_turns, float* out_scale) {
    if (!out_turns || !out_scale || rot < 2 || rot > 256 || rot % 2 || !(base > 1.0))
        return SPEC_ERR_INVALID_ARG;
    if (scaling < SPEC_ROPE_PLAIN || scaling > SPEC_ROPE_BY_PARTS) return SPEC_ERR_INVALID_ARG;
    if (scaling != SPEC_ROPE_PLAIN && !(factor >= 1.0)) return SPEC_ERR_INVALID_ARG;
    if (scaling == SPEC_ROPE_BY_PARTS && (!(original_len > 0.0) || !(fast > slow)))
        return SPEC_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925286766559;
    if (scaling == SPEC_ROPE_NTK) base *= std::pow(factor, double(rot) / std::max(1, rot - 2));
    for (int i = 0; i < rot / 2; ++i) {
        double th = std::pow(base, -2.0 * i / rot);
        if (scaling == SPEC_ROPE_LINEAR) th /= factor;
        if (scaling == SPEC_ROPE_BY_PARTS) {
            const double r = original_len * th / two_pi;
            const double g = std::min(1.0, std::max(0.0, (r - slow) / (fast - slow)));
            th *= (1.0 - g) / factor + g;
        }
        out_turns[i] = uint64_t(std::ldexp(th / two_pi, 64));  // th <= 1, so below 2^62
    }
    *out_scale = scaling == SPEC_ROPE_BY_PARTS ? float(0.1 * std::log(factor) + 1.0) : 1.f;
    return SPEC_OK;
}

spec_status spec_rope(const void* q, int q_heads, int64_t q_token_stride, int64_t q_head_stride,
                      void* out_q, int64_t oq_token_stride, int64_t oq_head_stride, const void* k,
                      int k_heads, int64_t k_token_stride, int64_t k_head_stride, void* out_k,
                      int64_t ok_token_stride, int64_t ok_head_stride, spec_dtype dtype, int D,
                      int64_t T, const int32_t* positions, const spec_rope_table* table,
                      int inverse, spec_stream_t stream) {
    if (T < 0 || q_heads < 0 || k_heads < 0 || q_heads > 65536 || k_heads > 65536 || D < 2 ||
        T > (1ll << 40) || !table)
        return SPEC_ERR_INVALID_ARG;
    if (dtype != SPEC_F32 && dtype != SPEC_BF16 && dtype != SPEC_F16) return SPEC_ERR_INVALID_ARG;
    if (D > 256 || D % 2) return SPEC_ERR_UNSUPPORTED;
    const spec_status ts = check_table(table, D);
    if (ts != SPEC_OK) return ts;
    if (T == 0 || q_heads + k_heads == 0) return SPEC_OK;
    if (!positions || (q_heads && (!q || !out_q)) || (k_heads && (!k || !out_k)))
        return SPEC_ERR_INVALID_ARG;
    const size_t es = dtype_bytes(dtype);
    if (!aligned(q, es) || !aligned(k, es) || !aligned(out_q, es) || !aligned(out_k, es) ||
        !aligned(positions, 4))
        return SPEC_ERR_UNSUPPORTED;
    RotArgs A = {};
    A.q = {q, out_q, q_token_stride, q_head_stride, oq_token_stride, oq_head_stride, q_heads};
    A.k = {k, out_k, k_token_stride, k_head_stride, ok_token_stride, ok_head_stride, k_heads};
    A.pos = positions;
    A.turns = reinterpret_cast<const unsigned long long*>(table->turns);
    A.half_rot = table->rot / 2;
    A.interleaved = table->layout == SPEC_ROPE_INTERLEAVED;
    A.scale = table->scale;
    A.sign = inverse ? -1.f : 1.f;
    A.D = D;
    A.T = T;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == SPEC_F32    ? launch_rotate_vec<float, false, PLAIN>(A, st)
                          : dtype == SPEC_BF16 ? launch_rotate_vec<__nv_bfloat16, false, PLAIN>(A, st)
                                               : launch_rotate_vec<__half, false, PLAIN>(A, st);
    return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

spec_status spec_kv_write(const spec_kv_cache* cache, const void* k, int64_t k_token_stride,
                          int64_t k_head_stride, const void* v, int64_t v_token_stride,
                          int64_t v_head_stride, spec_dtype dtype, int64_t T,
                          const int64_t* slots, const int32_t* positions,
                          const spec_rope_table* table, const void* q, int q_heads,
                          int64_t q_token_stride, int64_t q_head_stride, void* out_q,
                          int64_t oq_token_stride, int64_t oq_head_stride, int32_t* dev_status,
                          spec_stream_t stream) {
    const spec_status cs = check_cache(cache);
    if (cs != SPEC_OK) return cs;
    if (T < 0 || T > (1ll << 40) || q_heads < 0 || q_heads > 65536) return SPEC_ERR_INVALID_ARG;
    const bool e4 = cache->dtype == SPEC_E4M3;
    if (dtype != SPEC_F32 && dtype != SPEC_BF16 && dtype != SPEC_F16) return SPEC_ERR_INVALID_ARG;
    if (!e4 && int(dtype) != cache->dtype) return SPEC_ERR_INVALID_ARG;
    if (table) {
        const spec_status ts = check_table(table, cache->head_dim);
        if (ts != SPEC_OK) return ts;
        if (!positions && T > 0) return SPEC_ERR_INVALID_ARG;
    }
    if (q_heads && !table) return SPEC_ERR_INVALID_ARG;  // queries come along to be rotated
    if (T == 0) return SPEC_OK;
    if (!k || !v || !slots || (q_heads && (!q || !out_q))) return SPEC_ERR_INVALID_ARG;
    const size_t es = dtype_bytes(dtype);
    if (!aligned(k, es) || !aligned(v, es) || !aligned(q, es) || !aligned(out_q, es) ||
        !aligned(slots, 8) || !aligned(positions, 4) || !aligned(dev_status, 4))
        return SPEC_ERR_UNSUPPORTED;
    RotArgs A = {};
    if (q_heads)
        A.q = {q, out_q, q_token_stride, q_head_stride, oq_token_stride, oq_head_stride, q_heads};
    A.k = {k, nullptr, k_token_stride, k_head_stride, 0, 0, cache->heads};
    A.v = {v, nullptr, v_token_stride, v_head_stride, 0, 0, cache->heads};
    if (table) {
        A.pos = positions;
        A.turns = reinterpret_cast<const unsigned long long*>(table->turns);
        A.half_rot = table->rot / 2;
        A.interleaved = table->layout == SPEC_ROPE_INTERLEAVED;
        A.scale = table->scale;
    }
    A.sign = 1.f;
    A.D = cache->head_dim;
    A.T = T;
    A.c = view_of(*cache);
    A.slots = reinterpret_cast<const long long*>(slots);
    A.status = dev_status;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (e4)
        e = dtype == SPEC_F32    ? launch_rotate_vec<float, true, PLAIN>(A, st)
            : dtype == SPEC_BF16 ? launch_rotate_vec<__nv_bfloat16, true, PLAIN>(A, st)
                                 : launch_rotate_vec<__half, true, PLAIN>(A, st);
    else
        e = dtype == SPEC_BF16 ? launch_rotate_vec<__nv_bfloat16, false, PLAIN>(A, st)
                               : launch_rotate_vec<__half, false, PLAIN>(A, st);
    return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"

namespace {

template <typename C, typename T>
cudaError_t launch_read_to(const CacheView& c, int64_t T_, const int64_t* slots, void* out_k, void* out_v,
                           cudaStream_t st) {
    const long long n = T_ * c.heads * (c.D / (16 / int(sizeof(T))));
    const unsigned grid = unsigned(std::min<long long>((n + 255) / 256, 1ll << 22));
    const long long* s = reinterpret_cast<const long long*>(slots);
    T *k = static_cast<T*>(out_k), *v = static_cast<T*>(out_v);
    auto* kernel = n < (1ll << 31) && c.slots < (1ll << 32) ? k_kv_read<C, T, uint32_t> : k_kv_read<C, T, long long>;
    return launch_behind(kernel, dim3(grid), 256, 0, st, c, (long long)T_, s, k, v);
}
template <typename C>
cudaError_t launch_read(const CacheView& c, int64_t T, const int64_t* slots, int dtype,
                        void* out_k, void* out_v, cudaStream_t st) {
    if (dtype == SPEC_F32) return launch_read_to<C, float>(c, T, slots, out_k, out_v, st);
    if (dtype == SPEC_BF16) return launch_read_to<C, __nv_bfloat16>(c, T, slots, out_k, out_v, st);
    return launch_read_to<C, __half>(c, T, slots, out_k, out_v, st);
}

}  // namespace

extern "C" spec_status spec_kv_read(const spec_kv_cache* cache, int64_t T, const int64_t* slots,
                                    spec_dtype dtype, void* out_k, void* out_v,
                                    spec_stream_t stream) {
    const spec_status cs = check_cache(cache);
    if (cs != SPEC_OK) return cs;
    if (T < 0 || T > (1ll << 40)) return SPEC_ERR_INVALID_ARG;
    if (dtype != SPEC_F32 && dtype != SPEC_BF16 && dtype != SPEC_F16) return SPEC_ERR_INVALID_ARG;
    if (T == 0) return SPEC_OK;
    if (!slots || !out_k || !out_v) return SPEC_ERR_INVALID_ARG;
    if (!aligned(slots, 8) || !aligned(out_k, 16) || !aligned(out_v, 16))
        return SPEC_ERR_UNSUPPORTED;
    const CacheView c = view_of(*cache);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e =
        cache->dtype == SPEC_E4M3
            ? launch_read<uint8_t>(c, T, slots, dtype, out_k, out_v, st)
        : cache->dtype == SPEC_BF16
            ? launch_read<__nv_bfloat16>(c, T, slots, dtype, out_k, out_v, st)
            : launch_read<__half>(c, T, slots, dtype, out_k, out_v, st);
    return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
