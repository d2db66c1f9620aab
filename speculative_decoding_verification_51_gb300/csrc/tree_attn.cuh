// tree_attn.cuh -- attention of the drafted nodes over the paged cache: what
// the kernels share (arguments, the division of the work, the join of parts).
//
// The work is a list of items (request b, key head h, row tile r); a row is a
// (node, query head of the group) pair, row = node * G + head.  An item is
// ceil(length / TREE_TILE) tiles of tokens.  All tiles of all items, in
// order, are cut into as many equal shares as there are CTAs, so that ragged
// lengths load every SM alike.  A share's segment that holds a whole item
// writes its output; the others leave unnormalised sums with their reference
// and total in the workspace, and the CTA that arrives last joins an item's
// parts in order (the result does not depend on who that is).
#pragma once

#include <cuda.h>

#include "cache.cuh"

namespace sv {

struct AttnArgs {
    const void* q;
    long long qb, qn, qh;  // strides of q, elements
    void* out;
    float* lse;
    const int32_t* table;
    const uint32_t* masks;
    PlanView plan;
    const void* v;  // the cache's values (read again where some are not finite)
    const uint8_t* ks;
    const uint8_t* vs;
    long long v_page, v_head, v_token;
    int B, N, Hq, Hkv, G, D, page, max_pages;
    int rows, tiles_r;  // rows of a (request, key head), row tiles of them
    float c;            // scale * log2(e): scores are exponents of two
    int q_f16;          // q and out are f16 (else bf16)
    float* part_o;      // [2 * CTAs][R][width] unnormalised sums
    float* part_ml;     // [2 * CTAs][R][2] reference and total
    int32_t* status;
};

// A piece of one item that lies in this CTA's share.
struct Segment {
    int b, h, rt;
    int c0, c1;  // chunks of 16 tokens
    int t0, t1, tiles;  // tiles of the item: this piece's, and all
    int ctx, n;
    long long g;       // the piece's first tile in the list of all
};

struct Share {
    long long total, begin, end;
    int ctas;
};

__device__ __forceinline__ Share share_of(const AttnArgs& A) {
    Share s;
    s.total = (long long)A.plan.tiles[A.B] * A.Hkv * A.tiles_r;
    s.ctas = int(s.total < (long long)gridDim.x ? s.total : (long long)gridDim.x);
    s.begin = s.end = 0;
    if ((int)blockIdx.x < s.ctas) {
        s.begin = s.total * blockIdx.x / s.ctas;
        s.end = s.total * (blockIdx.x + 1) / s.ctas;
    }
    return s;
}
// the CTA whose share holds tile g
__device__ __forceinline__ int cta_of(const Share& s, long long g) {
    return int(((g + 1) * s.ctas - 1) / s.total);
}

// The request whose tiles hold g (a whole warp searches, 32 ways a step).
__device__ __forceinline__ int request_of(const AttnArgs& A, long long g) {
    const int lane = threadIdx.x & 31;
    const long long hr = (long long)A.Hkv * A.tiles_r;
    int lo = 0, hi = A.B;  // tiles[lo] * hr <= g < tiles[hi] * hr
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int i = lo + (lane + 1) * step;
        const bool le = i < hi && A.plan.tiles[i] * hr <= g;
        const int k = __popc(__ballot_sync(0xffffffffu, le));
        hi = min(hi, lo + (k + 1) * step);
        lo += k * step;
    }
    return lo;
}

// The segment that starts at tile g; b is the request that holds g or one before.
__device__ __forceinline__ Segment segment_at(const AttnArgs& A, const Share& s, long long g, int b) {
    const long long hr = (long long)A.Hkv * A.tiles_r;
    Segment x;
    int lo = A.plan.tiles[b], hi = A.plan.tiles[b + 1];
    while (hi * hr <= g) {
        ++b;
        lo = hi;
        hi = A.plan.tiles[b + 1];
    }
    x.b = b;
    x.g = g;
    x.tiles = hi - lo;
    const long long r = g - lo * hr;
    const int item = int(r / x.tiles);
    x.t0 = int(r - (long long)item * x.tiles);
    x.t1 = int(min((long long)x.tiles, x.t0 + (s.end - g)));
    x.h = item / A.tiles_r;
    x.rt = item - x.h * A.tiles_r;
    x.ctx = A.plan.ctx[b];
    x.n = A.plan.nodes[b];
    const int chunks = (x.ctx + x.n + 15) / 16;
    x.c0 = x.t0 * (TREE_TILE / 16);
    x.c1 = min(x.t1 * (TREE_TILE / 16), chunks);
    return x;
}

// ---------------------------------------------------------------- small pieces

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                            int w, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}

template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    uint32_t r;
    if constexpr (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// A value of the cache that is not finite: element (token t of request b, key
// head h, channel d), or 0 where it is finite.
template <int KIND>
__device__ __forceinline__ float not_finite_v(const AttnArgs& A, int b, int h, int t, int d) {
    const int p = A.table[(long long)b * A.max_pages + t / A.page];
    const long long at = p * A.v_page + h * A.v_head + (t % A.page) * A.v_token + d;
    float x;
    if constexpr (KIND == SPEC_E4M3) {
        const uint8_t u = static_cast<const uint8_t*>(A.v)[at];
        x = (u & 0x7f) == 0x7f ? __int_as_float(0x7fc00000) : 0.f;
    } else if constexpr (KIND == SPEC_F16) {
        x = __half2float(static_cast<const __half*>(A.v)[at]);
    } else {
        x = __bfloat162float(static_cast<const __nv_bfloat16*>(A.v)[at]);
    }
    return fabsf(x) < INFINITY ? 0.f : x;
}

__device__ __forceinline__ void store4(const AttnArgs& A, long long at, const float (&o)[4]) {
    uint2 w;
    if (A.q_f16) w = make_uint2(pack16<true>(o[0], o[1]), pack16<true>(o[2], o[3]));
    else w = make_uint2(pack16<false>(o[0], o[1]), pack16<false>(o[2], o[3]));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(A.out) + at) = w;
}

// One row's finished values: 4 channels from d on.
__device__ __forceinline__ void put_row(const AttnArgs& A, const Segment& s, int row, int d,
                                        const float (&o)[4], float total) {
    if (row >= A.rows || d >= A.D) return;
    const int v = row / A.G, g = row - v * A.G;
    const float f = v < s.n && total != 0.f ? 1.f / total : 0.f;
    const bool none = f == 0.f && !(total != total);
    float x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = none ? 0.f : o[e] * f;
    store4(A, (((long long)s.b * A.N + v) * A.Hq + s.h * A.G + g) * A.D + d, x);
}
__device__ __forceinline__ void put_lse(const AttnArgs& A, const Segment& s, int row, float ref,
                                        float total) {
    if (!A.lse || row >= A.rows) return;
    const int v = row / A.G, g = row - v * A.G;
    A.lse[((long long)s.b * A.N + v) * A.Hq + s.h * A.G + g] =
        v < s.n && total != 0.f ? (ref + log2f(total)) * 0.6931471805599453f : -INFINITY;
}

// After this CTA's part of an item lies in the workspace: the CTA that
// arrives last joins the parts (R rows of `width` channels each).
// `threads` threads call it together (tid their index), `sync` is their barrier
// and `flag` a shared word of theirs.
template <typename Sync>
__device__ __forceinline__ void join_parts(const AttnArgs& A, const Share& sh, const Segment& s,
                                           int R, int width, int* flag, int tid, int threads,
                                           Sync&& sync) {
    const long long g0 = s.g - s.t0;  // the item's first tile
    const int c0 = cta_of(sh, g0), c1 = cta_of(sh, g0 + s.tiles - 1);
    __threadfence();
    sync();
    if (tid == 0) {
        const int last = atomicAdd(&A.plan.arrived[c0], 1) == c1 - c0;
        if (last) A.plan.arrived[c0] = 0;  // as the next call finds it
        *flag = last;
    }
    sync();
    if (!*flag) return;
    __threadfence();
    const int quads = width / 4;
    for (int i = tid; i < R * quads; i += threads) {
        const int r = i / quads, d = (i - r * quads) * 4, row = s.rt * R + r;
        if (row >= A.rows) break;
        float ref = -INFINITY, total = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
        for (int c = c0; c <= c1; ++c) {
            const long long slot = 2 * c + (c == c0 ? 1 : 0);
            ref = fmaxf(ref, __ldcg(A.part_ml + (slot * R + r) * 2));
        }
        const float at = ref == -INFINITY ? 0.f : ref;
        for (int c = c0; c <= c1; ++c) {
            const long long slot = 2 * c + (c == c0 ? 1 : 0);
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(A.part_ml) + slot * R + r);
            const float4 x = __ldcg(reinterpret_cast<const float4*>(A.part_o + (slot * R + r) * width + d));
            const float f = ex2_approx(ml.x - at);
            total += f * ml.y;
            o[0] = fmaf(f, x.x, o[0]);
            o[1] = fmaf(f, x.y, o[1]);
            o[2] = fmaf(f, x.z, o[2]);
            o[3] = fmaf(f, x.w, o[3]);
        }
        put_row(A, s, row, d, o, total);
        if (d == 0) put_lse(A, s, row, ref, total);
    }
}
// the workspace slot of this CTA's part: the second where the item starts in
// its share (join_parts)
__device__ __forceinline__ long long part_slot(const Share& sh, const Segment& s) {
    return 2ll * blockIdx.x + (s.g - s.t0 >= sh.begin ? 1 : 0);
}

// Launchers (tree_attn_*.cu).
struct AttnLaunch {
    CUtensorMap mk, mv;
    AttnArgs A;
    int ctas;
    cudaStream_t st;
};
// mt: row tiles of 16 of k_attn_rows (1 or 2), or 0 for k_attn_tiles
cudaError_t launch_attn_bf16(const AttnLaunch& L, int mt);
cudaError_t launch_attn_f16(const AttnLaunch& L, int mt);
cudaError_t launch_attn_e4m3(const AttnLaunch& L, int mt);

}  // namespace sv
