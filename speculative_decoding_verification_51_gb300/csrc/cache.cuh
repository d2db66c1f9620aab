// cache.cuh -- shared by the operators around the verification (rope.cu,
// nodes.cu, tree_attn*.cu): element types, e4m3 rows, argument checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <initializer_list>
#include <utility>

#include "common.cuh"

namespace sv {

// ---------------------------------------------------------------- launches
// The operators' kernels are launched with programmatic dependent launch: a kernel's
// CTAs may take their SMs while the kernel before it in the stream ends.  A
// kernel lets the next one begin at once and waits for the end of the one before
// before it touches memory, in every CTA, so that ends follow in order.  Two differ:
// k_attn_join reads the plan ahead of its wait, lets nothing begin early and waits in
// one CTA at least; so the tile kernels, which it is launched behind, wait first and let
// it begin only then (were they to do as the others, it could read a plan that
// spec_tree_plan is still writing).  What one kernel costs behind another fell by 1.1 to
// 2.2 us: a step's four kernels for 256 trees took 41.0 us and take 32.2, one token's
// attention 10.3 and 8.5.
__device__ __forceinline__ void begin_after_previous() {
    griddep_launch_dependents();
    griddep_wait();
}
template <typename... P, typename... Q>
inline cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st,
                                 Q&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Q>(args)...);
}

// ---------------------------------------------------------------- elements

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// ---------------------------------------------------------------- e4m3 rows
// An e4m3 row holds x 2^-e with e the least integer for which max |x| <= 448
// 2^e.  A power of two shifts the exponent alone, so x 2^-e is exact and the
// value is rounded once; a scale of full precision would round twice and buy
// no accuracy, since e4m3 values have the same relative spacing in every
// binade but the lowest.

// e for a row's largest finite |x| (0 for a row of zeros: e = -126).
__device__ __forceinline__ int e4m3_exponent(float amax) {
    // 448 = 1.75 * 2^8: the mantissa of amax decides between two exponents
    const uint32_t u = __float_as_uint(amax);
    int e = int(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    // a subnormal amax is below 448 * 2^-126 all the same
    return e < -126 ? -126 : e;
}
// 2^e for e in [-126, 127]
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }
// x 2^-e, exact (e <= 120 for a float's exponent, so the factor is a float)
__device__ __forceinline__ float e4m3_scaled(float x, int e) { return x * exp2_int(-e); }
// |x| for the row maximum: infinities and NaN do not count
__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a < INFINITY ? a : 0.f;
}
// Two floats -> two e4m3 bytes (lo in bits 0..7), round to nearest even;
// infinities and NaN -> NaN.
__device__ __forceinline__ uint16_t pack_e4m3x2(float lo, float hi) {
    uint16_t r;
    // satfinite clamps infinities to 448, so they are made NaN first
    const float nan = __int_as_float(0x7fc00000);
    lo = fabsf(lo) < INFINITY ? lo : nan;
    hi = fabsf(hi) < INFINITY ? hi : nan;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two e4m3 bytes -> two halves (exact)
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
    return r;
}

// ---------------------------------------------------------------- a cache on the device

struct CacheView {
    void* k;
    void* v;
    uint8_t* ks;
    uint8_t* vs;
    long long page_stride, head_stride, token_stride;  // elements
    int page, heads, D, dtype;
    long long slots;  // num_pages * page
};

inline int dtype_bytes(int dt) {
    switch (dt) {
        case SPEC_F32: return 4;
        case SPEC_BF16:
        case SPEC_F16: return 2;
        case SPEC_E4M3: return 1;
    }
    return 0;
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
// (a null pointer is aligned)
inline bool all_aligned(size_t a, std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (!aligned(p, a)) return false;
    return true;
}

inline CacheView view_of(const spec_kv_cache& c) {
    CacheView v;
    v.k = c.k;
    v.v = c.v;
    v.ks = c.k_scale;
    v.vs = c.v_scale;
    v.page_stride = c.page_stride;
    v.head_stride = c.head_stride;
    v.token_stride = c.token_stride;
    v.page = c.page_size;
    v.heads = c.heads;
    v.D = c.head_dim;
    v.dtype = c.dtype;
    v.slots = (long long)c.num_pages * c.page_size;
    return v;
}

// The host-checkable part of a cache description.
inline spec_status check_cache(const spec_kv_cache* c) {
    if (!c || !c->k || !c->v) return SPEC_ERR_INVALID_ARG;
    if (c->dtype != SPEC_BF16 && c->dtype != SPEC_F16 && c->dtype != SPEC_E4M3)
        return SPEC_ERR_INVALID_ARG;
    if (c->num_pages < 1 || c->heads < 1 || c->head_dim < 1 || c->page_size < 1)
        return SPEC_ERR_INVALID_ARG;
    const bool e4 = c->dtype == SPEC_E4M3;
    if (e4 && (!c->k_scale || !c->v_scale)) return SPEC_ERR_INVALID_ARG;
    if (c->page_size % 16 || c->page_size > 65536) return SPEC_ERR_UNSUPPORTED;
    if (c->head_dim % (e4 ? 16 : 8) || c->head_dim > 256 || c->heads > 65535)
        return SPEC_ERR_UNSUPPORTED;
    const long long es = dtype_bytes(c->dtype);
    for (long long s : {(long long)c->page_stride, (long long)c->head_stride,
                        (long long)c->token_stride})
        if (s < 0 || (s * es) % 16 || s * es >= (1ll << 40)) return SPEC_ERR_UNSUPPORTED;
    if (c->token_stride < c->head_dim) return SPEC_ERR_INVALID_ARG;
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return SPEC_ERR_UNSUPPORTED;
    if (e4 && (!aligned(c->k_scale, 16) || !aligned(c->v_scale, 16))) return SPEC_ERR_UNSUPPORTED;
    return SPEC_OK;
}

// ---------------------------------------------------------------- a step's plan
// The plan buffer of spec_tree_plan (int32 words):
//   ctx[B], nodes[B]   the request's context and nodes (both 0: a bad request)
//   tiles[B + 1]       tiles of TREE_TILE tokens of the requests before b (a
//                      request has one tile at least, so that its rows are
//                      written)
// and zeros up to its end.  spec_tree_plan alone writes it.
constexpr int TREE_TILE = 128;

template <class I>
struct PlanLists {
    I* ctx;
    I* nodes;
    I* tiles;
};
using PlanView = PlanLists<const int>;
inline size_t plan_words(int B) { return size_t(B) * 3 + 1; }
template <class I>
inline PlanLists<I> plan_lists(I* plan, int B) {
    return {plan, plan + B, plan + 2 * size_t(B)};
}

// The device's SM count, read once per device.
int sm_count();

}  // namespace sv
