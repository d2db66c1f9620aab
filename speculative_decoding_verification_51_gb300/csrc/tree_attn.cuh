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
#include "tensor.cuh"

namespace sv {

struct AttnArgs {
    const void* q;
    long long qb, qn, qh;  // strides of q, elements
    void* out;
    float* lse;
    const int32_t* table;
    const uint32_t* masks;
    PlanView plan;
    unsigned long long* arrived;  // [CTAs] arrivals of the parts of the item that starts in a share (arrive)
    const void* v;  // the cache's values (read again where some are not finite)
    const uint8_t* ks;
    const uint8_t* vs;
    long long v_page, v_head, v_token;
    int B, N, Hq, Hkv, G, D, page, max_pages, num_pages;
    int rows, tiles_r;  // rows of a (request, key head), row tiles of them
    int box;            // tokens of one copy (k_attn_tiles)
    int lead;           // what an item costs beyond its tiles, in tiles
    float c;            // scale * log2(e): scores are exponents of two
    int q_f16;          // q and out are f16 (else bf16)
    float* part_o;      // [2 * CTAs][width / 4][R][4] unnormalised sums
    float* part_ml;     // [2 * CTAs][R][2] reference and total
    int32_t* status;
};

// A piece of one item that lies in this CTA's share.
struct Segment {
    int b, h, rt;
    int c0, c1;  // chunks of 16 tokens
    int t0, t1, tiles;  // tiles of the item: this piece's, and all
    int ctx, n;
    long long g;       // the piece's first tile's place in the list of all
};

// A page of the table, which spec_tree_plan found to be in the cache; one that was
// changed since then does not lead out of it.
__device__ __forceinline__ int page_in(const AttnArgs& A, int p) {
    return int(min(unsigned(p), unsigned(A.num_pages - 1)));
}

// A share is a stretch [begin, end) of the list of all items.  In the list an item
// takes its tiles' places and `lead` places before them: what it costs a CTA to
// turn to another item, in tiles (A.lead), so that CTAs with many short items get
// fewer tiles.  Nothing happens in a lead: a share's ends that fall into one are
// moved to its end and its beginning.  With less than a tile a CTA there is none (with
// leads there too such calls take 7 to 9% longer; with leads from one tile a CTA on
// instead of eight, those of 1 to 2 tiles 10% less, of 4 to 8 5%).
struct Share {
    long long total, begin, end;
    int ctas, lead;
};

// a / b and a % b, in 32 bits where they are enough
__device__ __forceinline__ long long quotient(long long a, long long b) {
    return (a | b) >> 32 ? a / b : (long long)(uint32_t(a) / uint32_t(b));
}
__device__ __forceinline__ long long remainder(long long a, long long b) {
    return (a | b) >> 32 ? a % b : (long long)(uint32_t(a) % uint32_t(b));
}

__device__ __forceinline__ Share share_of(const AttnArgs& A, int tiles) {
    const long long hr = (long long)A.Hkv * A.tiles_r;
    Share s;
    s.lead = tiles * hr >= (long long)gridDim.x ? A.lead : 0;
    s.total = (tiles + (long long)s.lead * A.B) * hr;
    s.ctas = int(s.total < (long long)gridDim.x ? s.total : (long long)gridDim.x);
    s.begin = s.end = 0;
    if ((int)blockIdx.x < s.ctas) {
        s.begin = quotient(s.total * blockIdx.x, s.ctas);
        s.end = quotient(s.total * (blockIdx.x + 1), s.ctas);
    }
    return s;
}

// The part of the plan's lists that a CTA starts with, in shared memory: their
// reads depend on one another, and each would wait for L2 or HBM.  Requests
// past the window are read where they lie.
constexpr int PLAN_WINDOW = 32;
struct PlanWindow {
    long long begin, end;  // the share's, moved out of leads
    int b0;
    int tiles[PLAN_WINDOW + 1], ctx[PLAN_WINDOW], nodes[PLAN_WINDOW];
};
struct Lists {
    const PlanWindow& w;
    const PlanView& p;
    int b0;
    __device__ __forceinline__ int tiles(int b) const {
        return b - b0 <= PLAN_WINDOW ? w.tiles[b - b0] : p.tiles[b];
    }
    __device__ __forceinline__ int ctx(int b) const { return b - b0 < PLAN_WINDOW ? w.ctx[b - b0] : p.ctx[b]; }
    __device__ __forceinline__ int nodes(int b) const {
        return b - b0 < PLAN_WINDOW ? w.nodes[b - b0] : p.nodes[b];
    }
};

// What request b (tiles lo to hi of the plan's list) says of a share: whether it
// holds its first place (then the window begins with request `b0`), and where its ends
// are moved to.
__device__ __forceinline__ void find_ends(const AttnArgs& A, PlanWindow& w, const Share& s, int b, int lo, int hi,
                                          int b0) {
    const long long hr = (long long)A.Hkv * A.tiles_r, from = (lo + (long long)s.lead * b) * hr;
    const int each = hi - lo + s.lead;
    const long long to = from + each * hr;
    if (from <= s.begin && s.begin < to) {
        w.b0 = b0;
        const long long into = remainder(s.begin - from, each);
        w.begin = s.begin + max(s.lead - into, 0ll);
    }
    if (from < s.end && s.end <= to) {  // (the end of an item is one already)
        const long long into = remainder(s.end - from, each);
        w.end = s.end - (into <= s.lead ? into : 0ll);
    }
}

// This CTA's share, and the window from the request that holds its first tile
// on.  Call with the whole CTA; false (for all of it) where there is no share.
__device__ __forceinline__ bool read_plan(const AttnArgs& A, PlanWindow& w, Share& s) {
    if (A.B <= PLAN_WINDOW) {  // the window holds every request: one round of reads
        if (int(threadIdx.x) <= A.B) {
            w.tiles[threadIdx.x] = A.plan.tiles[threadIdx.x];
            if (int(threadIdx.x) < A.B) {
                w.ctx[threadIdx.x] = A.plan.ctx[threadIdx.x];
                w.nodes[threadIdx.x] = A.plan.nodes[threadIdx.x];
            }
        }
        if (threadIdx.x == 0) w.b0 = 0;
        __syncthreads();
        s = share_of(A, w.tiles[A.B]);
        if (s.begin >= s.end || !s.lead) return s.begin < s.end;
        if (int(threadIdx.x) < A.B) find_ends(A, w, s, threadIdx.x, w.tiles[threadIdx.x], w.tiles[threadIdx.x + 1], 0);
        __syncthreads();
        s.begin = w.begin;
        s.end = w.end;
        return s.begin < s.end;
    }
    const int last = A.plan.tiles[A.B];
    bool any = false;
    for (int i = threadIdx.x; i < A.B; i += blockDim.x) {
        const int lo = A.plan.tiles[i], hi = A.plan.tiles[i + 1];
        if (!any) {
            s = share_of(A, last);
            any = true;
        }
        find_ends(A, w, s, i, lo, hi, i);
    }
    s = share_of(A, last);
    if (s.begin >= s.end) return false;
    __syncthreads();
    s.begin = w.begin;
    s.end = w.end;
    const int b0 = w.b0;
    for (int i = threadIdx.x; i <= PLAN_WINDOW && b0 + i <= A.B; i += blockDim.x) {
        w.tiles[i] = A.plan.tiles[b0 + i];
        if (i < PLAN_WINDOW && b0 + i < A.B) {
            w.ctx[i] = A.plan.ctx[b0 + i];
            w.nodes[i] = A.plan.nodes[b0 + i];
        }
    }
    __syncthreads();
    return s.begin < s.end;
}

// the CTA whose share holds place g
__device__ __forceinline__ int cta_of(const Share& s, long long g) {
    return int(quotient((g + 1) * s.ctas - 1, s.total));
}

// The segment that starts at place g (a tile, or the lead before an item's first
// one); b is the request that holds g or one before.
__device__ __forceinline__ Segment segment_at(const AttnArgs& A, const Lists& L, const Share& s, long long g, int b) {
    const long long hr = (long long)A.Hkv * A.tiles_r;
    Segment x;
    int lo = L.tiles(b), hi = L.tiles(b + 1);
    while ((hi + (long long)s.lead * (b + 1)) * hr <= g) {
        ++b;
        lo = hi;
        hi = L.tiles(b + 1);
    }
    x.b = b;
    x.tiles = hi - lo;
    const int each = x.tiles + s.lead;
    const long long r = g - (lo + (long long)s.lead * b) * hr;
    const int item = int(quotient(r, each));
    const int at = int(r - (long long)item * each) - s.lead;
    x.t0 = max(at, 0);
    x.g = g + (x.t0 - at);
    x.t1 = int(min((long long)x.tiles, x.t0 + (s.end - x.g)));
    x.h = item / A.tiles_r;
    x.rt = item - x.h * A.tiles_r;
    x.ctx = L.ctx(b);
    x.n = L.nodes(b);
    const int chunks = (x.ctx + x.n + 15) / 16;
    x.c0 = x.t0 * (TREE_TILE / 16);
    x.c1 = min(x.t1 * (TREE_TILE / 16), chunks);
    return x;
}

// ---------------------------------------------------------------- small pieces

// A value of the cache that is not finite: element (token t of request b, key
// head h, channel d), or 0 where it is finite.
template <int KIND>
__device__ __forceinline__ float not_finite_v(const AttnArgs& A, int b, int h, int t, int d) {
    const int p = page_in(A, A.table[(long long)b * A.max_pages + t / A.page]);
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

// One row's finished values: 4 channels from d on.  Zeros for a node past the
// tree (its row ran over the context too, so that its sums and total may be NaN)
// and for a row that saw nothing; NaN where the total is.
__device__ __forceinline__ void put_row(const AttnArgs& A, const Segment& s, int row, int d,
                                        const float (&o)[4], float total) {
    if (row >= A.rows || d >= A.D) return;
    const int v = row / A.G, g = row - v * A.G;
    const bool none = v >= s.n || total == 0.f;
    const float f = none ? 0.f : 1.f / total;
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

// Counts an arrival at `w` and says whether it is the last of `parts`.  The workspace may
// hold anything before its first use, so that a count is one only beneath a mark of
// 48 bits (memory that holds the mark by chance would be taken for a count).  An
// arrival that finds no mark has not counted: it puts the mark there with itself as the
// first, or counts beneath the one that another put there meanwhile; every retry means
// that another arrival went on.  Whoever is last puts the count back to zero, so that
// later calls need one atomic.
constexpr unsigned long long ARRIVED = 0x51c2e98a437dull << 16;
__device__ __forceinline__ bool arrive(unsigned long long* w, int parts) {
    constexpr unsigned long long COUNT = 0xffff;
    unsigned long long old = atomicAdd(w, 1ull);
    while ((old & ~COUNT) != ARRIVED) {
        const unsigned long long now = atomicAdd(w, 0ull);
        if ((now & ~COUNT) == ARRIVED) {
            old = atomicAdd(w, 1ull);
        } else if (atomicCAS(w, now, ARRIVED | 1ull) == now) {
            old = ARRIVED;
        }
    }
    const bool last = int(old & COUNT) + 1 == parts;
    if (last) *w = ARRIVED;
    return last;
}

// After this CTA's part of an item lies in the workspace: the CTA that
// arrives last joins the parts (R rows of `width` channels each).
// `threads` threads call it together (tid their index, `bar` their barrier) and
// `flag` is a shared word of theirs.
template <int U>
__device__ __forceinline__ void join_parts(const AttnArgs& A, const Share& sh, const Segment& s,
                                           int R, int width, int* flag, int tid, int threads,
                                           int bar) {
    auto sync = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(threads) : "memory"); };
    const long long g0 = s.g - s.t0;  // the item's first tile
    const int c0 = cta_of(sh, g0), c1 = cta_of(sh, g0 + s.tiles - 1);
    __threadfence();
    sync();
    if (tid == 0) *flag = arrive(A.arrived + c0, c1 - c0 + 1);
    sync();
    if (!*flag) return;
    __threadfence();
    // A thread keeps one row (R divides the number of threads) and takes U groups
    // of 4 channels at a time, 8 parts of each in flight; the lanes' rows lie side
    // by side, so that every read is coalesced.
    const int r = tid % R, row = s.rt * R + r, parts = c1 - c0 + 1, step = threads / R;
    auto slot = [&](int c) { return 2ll * (c0 + c) + (c == 0 ? 1 : 0); };
    const float2* ml = reinterpret_cast<const float2*>(A.part_ml) + r;
    const int quads = width / 4;
    for (int q = tid / R; q < quads; q += U * step) {
        float ref = -INFINITY, total = 0.f, o[U][4] = {};
        for (int c = 0; c < parts; c += 8) {  // running sums, by the running reference
            float2 z[8];
            float4 x[8][U];
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                z[y] = c + y < parts ? __ldcg(ml + slot(c + y) * R) : make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    x[y][u] = c + y < parts && q + u * step < quads
                                  ? __ldcg(reinterpret_cast<const float4*>(A.part_o) + (slot(c + y) * quads + q + u * step) * R + r)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float to = ref;
#pragma unroll
            for (int y = 0; y < 8; ++y) to = fmaxf(to, z[y].x);
            const float at = to == -INFINITY ? 0.f : to, f = ex2_approx(ref - at);
            ref = to;
            total *= f;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[u][e] *= f;
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                const float w = ex2_approx(z[y].x - at);  // 0 for a part that is not there
                total = fmaf(w, z[y].y, total);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    o[u][0] = fmaf(w, x[y][u].x, o[u][0]);
                    o[u][1] = fmaf(w, x[y][u].y, o[u][1]);
                    o[u][2] = fmaf(w, x[y][u].z, o[u][2]);
                    o[u][3] = fmaf(w, x[y][u].w, o[u][3]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (q + u * step < quads) put_row(A, s, row, (q + u * step) * 4, o[u], total);
        if (q == 0) put_lse(A, s, row, ref, total);
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
// k_attn_tiles leaves the parts of items to k_attn_join, launched behind it
// (tree_attn.cu); rows of `width` channels.
cudaError_t launch_attn_join(const AttnLaunch& L, int width);
// by k_attn_tiles, or k_attn_rows
cudaError_t launch_attn_bf16(const AttnLaunch& L, bool tiles);
cudaError_t launch_attn_f16(const AttnLaunch& L, bool tiles);
cudaError_t launch_attn_e4m3(const AttnLaunch& L, bool tiles);

}  // namespace sv
