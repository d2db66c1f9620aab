// tree_attn_tiles_e4m3.cuh -- k_attn_tiles_e4m3: k_attn_tiles over an 8-bit cache.
//
// 32 trees of 32 nodes (128 rows a key head) over 1000 to 16384 tokens take 197 us: 0.45
// of the measured copy rate and 0.30 of the tensor rate.  What bounds it is a
// tile's softmax, some twice the 1050 cycles that HBM would need.
//
// An SM's shared memory moves 128 bytes a cycle, and over an 8-bit cache that is
// what runs out first: a tile of 128 tokens (32 KB) has some 1400 cycles to
// match HBM.  So K's bytes are the operand as they lie, and only V becomes
// 16-bit (bytes in by TMA 32 KB, V read 16 and written 32 as f16, operands read
// 64-96 + 32).  Weights are an operand in TMEM; queries lie in shared memory, since TMEM
// has room for two tiles' scores and weights and the sums, and no more.
//
// Scores.  Products of 8-bit types (kind::f8f6f4) take queries of 8 bits, split: q 2^-a
// = h1 + h2 (+ h3), h1 = e4m3(q 2^-a) with 4 significant bits, then e5m2 terms of what
// is left, with 3 (the remainder's sign gives one more), a power of two a row that
// brings the largest to 448 or less.  Two terms hold bf16's 8 bits, three f16's 11.
// A value so small that h1 falls among e4m3's last steps of 2^-9 leaves a remainder
// of 2^-10 at most, of which e5m2 (steps down to 2^-16) keeps 3 bits: two terms
// are off by 2^-14 and three by 2^-17, 2^-21.8 and 2^-24.8 of the row's largest value.
// (e4m3 terms throughout: 2^-17.8.)  The terms' products add up in one accumulator.
// K's scale comes afterwards: a tile's scale bytes are turned to
// factors, and the exponent of a weight is (s rc) ck[t] - m.
//
// Values.  Where the exponents of a tile's rows lie within 8 of one another, v 2^e is
// stored as f16 v 2^(e - E), E the largest of them: exact.  2^E joins the exponents of the
// tile's weights, w_t = 2^(s_t + E - m), so that all tiles' sums are in one unit; the
// total takes 2^-E times the tile's weights.  In any other tile (rows of zeros have
// the least exponent there is, so theirs are such tiles) E could be one that a row
// does not see, or that of a token of no weight, and would take the bits of all the
// others: there the values stay as they lie and w_t = 2^(s_t + e_t - m), with a second
// exponential for the total.  (That path for every tile takes the trees above 293 us
// instead of 197.)  E and e_t are taken as -92 or more in m, so that zeros do not push
// the total out of float32.
//
// Weights are f16.  A raised reference leaves the largest at 2^8 or less, and they
// may grow to 2^15: so 8 octaves that E may exceed a row's own exponents by, or the
// tail of a long context 2^25 times below its largest weight, still count.
//
// Softmax.  Two threads a row, each half of the tile's tokens, since one warp a
// scheduler leaves it idle most of the time.  They keep one reference, which is
// raised seldom: a vote of the two warps says whether any row's weights are too
// large, and only then are its largest exponent found and the weights made again.
//
// Warps: 0 and 2 copies; 1 products with K; 3 products with V; 4..7 and 8..11 softmax;
// 12..19 V, and K's factors.
#pragma once

#include "tree_attn_tiles.cuh"

namespace sv {

template <int DP>
struct TilesE4Shape {
    static constexpr int HALVES = DP / 64;
    static constexpr int OPERAND = HALVES * 16384;  // 128 tokens of f16 channels
    static constexpr int RAW = 16384, RAWS = 3;     // 128 tokens (or rows) of 128 bytes
    static constexpr size_t SMEM = 1024 + size_t(RAWS) * 2 * RAW + 2 * OPERAND + 3 * RAW;
    static_assert(SMEM + 12288 <= 232448, "shared memory");
    static constexpr int THREADS = 640;
};

// D f32, A e4m3 (or e5m2: bit 7), B e4m3, both K-major, M = N = 128
constexpr int AT_SPREAD = 8;               // exponents of one tile's values that one unit serves
constexpr int AT_WIDE = 1 << 20;           // in place of the unit: the values have exponents of their own
constexpr float AT_TOP = 8.f, AT_LEAST = -92.f;
constexpr uint32_t AT_ID_E4 = (1u << 4) | (uint32_t(128 >> 3) << 17) | (uint32_t(128 >> 4) << 24);
__device__ __forceinline__ void at_mma_e4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// 2^d as two halves (d <= 0; 0 below f16's least subnormal)
__device__ __forceinline__ uint32_t half2_exp2(int d) {
    const uint32_t h = d >= -14 ? uint32_t(d + 15) << 10 : d >= -24 ? 1u << (d + 24) : 0u;
    return h * 0x10001u;
}
__device__ __forceinline__ uint32_t half2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// 4 columns of this thread's lane, and 2 of them written
__device__ __forceinline__ void at_ld4(uint32_t t, uint32_t (&r)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(t));
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3])::"memory");
}
__device__ __forceinline__ void at_st2(uint32_t t, const uint32_t (&r)[2]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(t), "r"(r[0]), "r"(r[1]) : "memory");
}
// 2^-d for a whole d >= 0 (0 where it is no normal float)
__device__ __forceinline__ float exp2_down(float d) { return d < 127.f ? exp2_int(-int(d)) : 0.f; }
// The first or a later term of two halves: their e4m3 or e5m2 bytes; the halves keep
// what is left (a difference of neighbours, so exact).
template <bool FIRST>
__device__ __forceinline__ uint32_t query_term(uint32_t& x) {
    uint16_t w;
    uint32_t h;
    if constexpr (FIRST) {
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(w) : "r"(x));
        h = e4m3x2_to_f16x2(w);
    } else {
        asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(w) : "r"(x));
        asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(w));
    }
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(x) : "r"(h));
    return w;
}

template <int DP>
__global__ void __launch_bounds__(TilesE4Shape<DP>::THREADS, 1)
    k_attn_tiles_e4m3(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                      const __grid_constant__ AttnArgs A) {
    using S = TilesE4Shape<DP>;
    constexpr int NR = S::RAWS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    uint8_t* sm_raw = smem;                     // [raws][K, V][128 tokens][128]
    uint8_t* sm_v = smem + NR * 2 * S::RAW;     // [2] f16 values
    uint8_t* sm_q = sm_v + 2 * S::OPERAND;      // [terms][128 rows][128] queries
    __shared__ __align__(16) uint8_t sm_sc[NR * 256];     // scale bytes
    __shared__ __align__(16) float sm_ck[2][128];         // K's factors
    __shared__ __align__(16) float sm_ve[2][128];         // V's exponents, in a tile that has no unit
    __shared__ __align__(8) uint64_t rkf[NR], rke[NR], rvf[NR], rve[NR], vf[2], ve[2];
    __shared__ __align__(8) uint64_t sf[2], pf[2], pv[2], qf, of, fin[2];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag, unit_v[2];
    __shared__ uint32_t bad_nodes[2];
    __shared__ float2 sm_max[2][128];          // what the halves of a row exchange: queries,
    __shared__ float sm_ref[2][128], sm_tot[2][128];  // references, totals
    __shared__ PlanWindow window;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // in this order: k_attn_join, which begins next, reads the plan before its own wait
    griddep_wait();
    griddep_launch_dependents();
    Share share;
    if (!read_plan(A, window, share)) return;  // the whole CTA
    const int first = window.b0;
    const Lists L = {window, A.plan, first};
    if (threadIdx.x == 0) {
        for (int i = 0; i < NR; ++i) {
            mbar_init(&rkf[i], 1);
            mbar_init(&rke[i], 2);  // the products, and the factors
            mbar_init(&rvf[i], 1);
            mbar_init(&rve[i], 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&vf[i], 8);
            mbar_init(&ve[i], 1);
            mbar_init(&sf[i], 1);
            mbar_init(&pf[i], 8);
            mbar_init(&pv[i], 1);
        }
        mbar_init(&qf, 8);
        mbar_init(&of, 8);
        mbar_init(&fin[0], 1);
        mbar_init(&fin[1], 1);
        abort_flag = 0;
        bad_nodes[0] = bad_nodes[1] = 0;
        fence_mbarrier_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_u32(&tmem_base))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    at_before();
    __syncthreads();
    at_after();
    const uint32_t tbase = tmem_base;
    // S at 0 and 128, O, P at 384 and 448
    constexpr uint32_t T_O = 256, T_P = 384;
    const int terms = A.q_f16 ? 3 : 2;
    volatile int* gone = &abort_flag;
    // a bounded wait; once one has run out nobody waits any more
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity & 1u) || *gone) return;
        if (!at_wait_bounded(bar, parity & 1u, AT_WAIT_NS)) *gone = 1;
    };

    // registers from the other warpgroups to softmax (64 + 2 * 136 + 2 * 72 <= 5 * 96):
    // in 96 its columns spill, to an L1 that shared memory has left little of
    if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp >= 12) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 0 || warp == 2) {
        // ---- copies of K (warp 0) and V (warp 2; together they would be late: a copy
        // takes some 100 cycles to issue): lane = (rows or scales, box of A.box tokens)
        const int side = warp >> 1;
        uint64_t *full = side ? rvf : rkf, *empty = side ? rve : rke;
        const CUtensorMap* map = side ? &mv : &mk;
        const uint8_t* scales = side ? A.vs : A.ks;
        const int chunk = lane & 7, part = lane >> 3, boxes = 128 / A.box;
        const uint32_t box_bytes = uint32_t(A.box) * 128;
        uint32_t i = 0;  // tiles so far
        int b_at = first;
        for (long long g = share.begin; g < share.end;) {
            const Segment s = segment_at(A, L, share, g, b_at);
            b_at = s.b;
            g = s.g + s.t1 - s.t0;
            const int len = s.ctx + s.n;
            const int32_t* table = A.table + (long long)s.b * A.max_pages;
            auto page_of = [&](int t, int& off) {
                const int tok = t * 128 + chunk * A.box;
                off = -1;  // no box for this lane
                if (t >= s.t1 || chunk >= boxes || tok >= len) return 0;
                const int p = tok / A.page;
                off = tok - p * A.page;
                return __ldg(table + p);  // (nothing is done with it before the next tile: it takes long)
            };
            int off, page = page_of(s.t0, off);
            for (int t = s.t0; t < s.t1; ++t, ++i) {
                const int nv = min(boxes, max(0, (len - t * 128 + A.box - 1) / A.box));
                int off2;
                const int page2 = page_of(t + 1, off2);
                const uint32_t st = i % NR, ph = i / NR;
                const int in = page_in(A, page);
                if (lane == 0) {
                    wait(&empty[st], ph ^ 1u);
                    if (!*gone) mbar_arrive_expect_tx(&full[st], nv * (box_bytes + A.box));
                }
                __syncwarp();
                if (off >= 0 && !*gone) {
                    if (part == 0)
                        tma_load_4d(sm_raw + (st * 2 + side) * S::RAW + chunk * box_bytes, map, 0, off, s.h, in, &full[st]);
                    if (part == 1)
                        bulk_g2s(sm_sc + st * 256 + side * 128 + chunk * A.box,
                                 scales + ((long long)in * A.Hkv + s.h) * A.page + off, A.box, &full[st]);
                }
                page = page2;
                off = off2;
            }
        }
        // every copy has landed before the CTA leaves (they have, unless a wait ran out)
        if (lane == 0 && *gone) {
            for (uint32_t j = i > NR ? i - NR : 0; j < i; ++j)
                at_wait_bounded(&full[j % NR], (j / NR) & 1u, AT_WAIT_NS / 8);
        }
    } else if (warp == 1) {
        // ---- products with K
        if (lane == 0) {
            uint32_t j = 0, seg = 0;
            int b_at = first;
            for (long long g = share.begin; g < share.end; ++seg) {
                const Segment s = segment_at(A, L, share, g, b_at);
                b_at = s.b;
                g = s.g + s.t1 - s.t0;
                wait(&qf, seg);
                for (int t = s.t0; t < s.t1; ++t, ++j) {
                    const uint32_t rs = j % NR;
                    wait(&rkf[rs], j / NR);
                    if (j >= 2) wait(&pf[j & 1], (j - 2) >> 1);  // those of tile j - 2 are weights
                    at_after();
                    const uint32_t ka = smem_u32(sm_raw) + rs * 2 * S::RAW, qa = smem_u32(sm_q);
                    for (int x = 0; x < terms; ++x)
#pragma unroll
                        for (int k = 0; k < DP / 32; ++k)
                            at_mma_e4(tbase + (j & 1) * 128, at_desc_k(qa + x * S::RAW + k * 32), at_desc_k(ka + k * 32),
                                      AT_ID_E4 | (x ? 1u << 7 : 0u), x > 0 || k > 0);
                    at_commit(&sf[j & 1]);
                    at_commit(&rke[rs]);
                }
            }
            at_commit(&fin[0]);  // every product is done before TMEM is freed
            at_wait_bounded(&fin[0], 0, AT_WAIT_NS);
        }
    } else if (warp == 3) {
        // ---- products with V, from a thread of their own: either's waits and commits
        // (some 100 cycles each) would keep the other's products from being issued
        if (lane == 0) {
            constexpr uint32_t id_o = at_idesc<true>(DP, true);
            uint32_t i = 0, seg = 0;
            int b_at = first;
            for (long long g = share.begin; g < share.end; ++seg) {
                const Segment s = segment_at(A, L, share, g, b_at);
                b_at = s.b;
                g = s.g + s.t1 - s.t0;
                for (int t = s.t0; t < s.t1; ++t, ++i) {
                    wait(&vf[i & 1], i >> 1);
                    wait(&pf[i & 1], i >> 1);
                    if (t == s.t0) wait(&of, seg ^ 1u);  // the last segment's rows have been read
                    at_after();
                    const uint32_t va = smem_u32(sm_v) + (i & 1) * S::OPERAND;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        at_mma_ts(tbase + T_O, tbase + T_P + (i & 1) * 64 + k * 8, at_desc_mn(va + k * 2048), id_o,
                                  t > s.t0 || k > 0);
                    at_commit(&pv[i & 1]);
                    at_commit(&ve[i & 1]);
                }
            }
            at_commit(&fin[1]);
            at_wait_bounded(&fin[1], 0, AT_WAIT_NS);
        }
    } else if (warp >= 4 && warp < 12) {
        // ---- softmax: row = this thread's TMEM lane, tokens (and channels) of one half
        asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
        const int half = (warp - 4) >> 2, w = warp & 3, r = w * 32 + lane, tid = r;
        const uint32_t lanes = uint32_t(w * 32) << 16;
        constexpr int CH = DP / 2;  // channels of a half
        const float c = fabsf(A.c), sign = A.c < 0.f ? -1.f : 1.f;
        auto sync = [&]() { asm volatile("bar.sync 1, 256;" ::: "memory"); };
        // the two warps of 32 rows
        auto sync_rows = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(2 + w) : "memory"); };
        auto any_of_rows = [&](bool p) {
            uint32_t any;
            asm volatile(
                "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                "bar.red.or.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                : "=r"(any)
                : "r"(uint32_t(p)), "r"(2 + w)
                : "memory");
            return any != 0;
        };
        float rc = 0.f;  // the row's factor on scores
        auto load_q = [&](const Segment& s) {
            const int row = s.rt * 128 + r, v = row / A.G;
            const bool on = row < A.rows && v < s.n;
            const uint16_t* src = static_cast<const uint16_t*>(A.q) + s.b * A.qb + v * A.qn +
                                  (s.h * A.G + row - v * A.G) * A.qh + half * CH;
            uint4 u[CH / 8];  // every load in flight at once
#pragma unroll
            for (int j = 0; j < CH / 8; ++j)
                u[j] = on && half * CH + j * 8 < A.D ? __ldg(reinterpret_cast<const uint4*>(src + j * 8)) : make_uint4(0, 0, 0, 0);
            auto pair = [&](uint32_t x) {
                return A.q_f16 ? __half22float2(*reinterpret_cast<const __half2*>(&x)) : make_float2(bf16_lo(x), bf16_hi(x));
            };
            float m = 0.f, odd = 0.f;  // odd: NaN where some value is not finite
#pragma unroll
            for (int j = 0; j < CH / 8; ++j) {
                const uint32_t x[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = pair(x[e]);
                    m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
                    odd = fmaf(f.x, 0.f, fmaf(f.y, 0.f, odd));
                }
            }
            sm_max[half][r] = make_float2(m, odd);
            sync_rows();
            m = fmaxf(m, sm_max[half ^ 1][r].x);
            odd += sm_max[half ^ 1][r].y;
            // (then the row's scores are NaN, by its operand: by its factor the -inf of what it
            // does not see would be, too)
            const bool bad = !(odd == 0.f);
            const int ex = bad ? 0 : e4m3_exponent(m);
            const float down = bad ? __int_as_float(0x7fc00000) : exp2_int(-ex) * sign;
            // a factor of zero would make NaN of -inf; no score of this size counts
            rc = fmaxf(c * exp2_int(ex), 1e-30f);
#pragma unroll
            for (int j = 0; j < CH / 32; ++j) {
                // as halves: 11 bits, and below 2^-14 of the scale steps of 2^-24
                uint32_t f[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const uint4& y = u[j * 4 + e / 4];
                    const float2 z = pair(e % 4 == 0 ? y.x : e % 4 == 1 ? y.y : e % 4 == 2 ? y.z : y.w);
                    f[e] = pack16<true>(z.x * down, z.y * down);
                }
#pragma unroll
                for (int x = 0; x < 3; ++x) {
                    if (x == 2 && !A.q_f16) break;
                    uint32_t o[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (x == 0) o[e] = query_term<true>(f[2 * e]) | query_term<true>(f[2 * e + 1]) << 16;
                        else o[e] = query_term<false>(f[2 * e]) | query_term<false>(f[2 * e + 1]) << 16;
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *reinterpret_cast<uint4*>(sm_q + x * S::RAW + r * 128 + ((((half * CH + j * 32) / 16 + e) ^ (r & 7)) << 4)) =
                            make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) at_arrive(&qf);
        };
        uint32_t i = 0, seg = 0;
        Segment s = segment_at(A, L, share, share.begin, first);
        load_q(s);
        for (;; ++seg) {
            const int row = s.rt * 128 + r, node = row / A.G;
            uint32_t mask = 0;
            if (row < A.rows && node < s.n)
                mask = A.masks[(long long)s.b * A.N + node] & (0xffffffffu >> (32 - s.n));
            float ref = -INFINITY, tot = 0.f;
            // the segment after this one; its query row comes to L2 meanwhile
            const long long next = s.g + (s.t1 - s.t0);
            const bool more = next < share.end;
            Segment after = s;
            if (more) {
                after = segment_at(A, L, share, next, s.b);
                const int nr = after.rt * 128 + r, nv = nr / A.G;
                if (nr < A.rows && nv < after.n) {
                    const uint16_t* src = static_cast<const uint16_t*>(A.q) + after.b * A.qb + nv * A.qn +
                                          (after.h * A.G + nr - nv * A.G) * A.qh;
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(src));
                    if (A.D > 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + 64));
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(A.masks + (long long)after.b * A.N + nv));
                }
            }
            for (int t = s.t0; t < s.t1; ++t, ++i) {
                const uint32_t sa = tbase + lanes + (i & 1) * 128 + half * 64;
                const uint32_t pa = tbase + lanes + T_P + (i & 1) * 64 + half * 32;
                const int t0 = t * 128;
                const bool tail = t0 + 128 > s.ctx;
                {   // waits side by side: each costs some 100 cycles though it is over.
                    // (V being there says that the products of tile i - 2, whose
                    // weights lay where this one's will, are done)
                    const bool w0 = mbar_try_wait(&sf[i & 1], i >> 1 & 1), w1 = mbar_try_wait(&vf[i & 1], i >> 1 & 1);
                    if (!w0) wait(&sf[i & 1], i >> 1);
                    if (!w1) wait(&vf[i & 1], i >> 1);
                }
                at_after();
                if (__builtin_expect(tail, 0)) hide_unseen(sa, t0 + half * 64 - s.ctx, mask, 64);
                const int unit_i = unit_v[i & 1];
                const bool wide = unit_i == AT_WIDE;
                const float unit = wide ? 0.f : float(unit_i);
                const float* ve = sm_ve[i & 1] + half * 64;
                const float4* ck = reinterpret_cast<const float4*>(sm_ck[i & 1] + half * 64);
                const uint64_t rc2 = f2_pack(rc, rc);
                // exponents of tokens j .. j + 31 by `base`, in place of their scores
                auto exponents = [&](uint32_t (&x)[32], int j, float base) {
                    at_ld32(sa + j, x);
                    const uint64_t at2 = f2_pack(unit - base, unit - base);
                    at_ld_wait(x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float4 k4 = ck[j / 4 + e];
                        float a, b;
                        f2_unpack(f2_fma(f2_mul(f2_pack(__uint_as_float(x[4 * e]), __uint_as_float(x[4 * e + 1])), rc2),
                                         f2_pack(k4.x, k4.y), at2), a, b);
                        x[4 * e] = __float_as_uint(a);
                        x[4 * e + 1] = __float_as_uint(b);
                        f2_unpack(f2_fma(f2_mul(f2_pack(__uint_as_float(x[4 * e + 2]), __uint_as_float(x[4 * e + 3])), rc2),
                                         f2_pack(k4.z, k4.w), at2), a, b);
                        x[4 * e + 2] = __float_as_uint(a);
                        x[4 * e + 3] = __float_as_uint(b);
                    }
                };
                // (a tile without a unit, 4 tokens at a time: as many as above would take so much of the
                // instruction cache that all tiles wait; 32 rows over 1000 to 16384 tokens 185 us
                // instead of 195)
                auto exponent = [&](uint32_t x, const float4& k4, int e, float base) {
                    return fmaf(__uint_as_float(x) * rc, e == 0 ? k4.x : e == 1 ? k4.y : e == 2 ? k4.z : k4.w, -base);
                };
                // The weights by the reference as it is.  None is above 2^15 where their
                // sum is not; where some row's sum is (or it has no reference yet), its
                // reference is raised to the largest exponent less 8 and they are made again.
                // (So also where 2^(s_t - m), of which a tile without a unit has the sum `all`,
                // nears float32's limit: zeros with all the weight.)
                float s0, s1, all = 0.f;
                for (bool again = false;; again = true) {
                    const float base = ref == -INFINITY ? 0.f : ref;
                    uint64_t sum = f2_pack(0.f, 0.f);
                    if (__builtin_expect(!wide, 1)) {
#pragma unroll 1
                        for (int j = 0; j < 64; j += 32) {
                            uint32_t x[32], p[16];
                            exponents(x, j, base);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float a = ex2_approx(__uint_as_float(x[2 * e])), b = ex2_approx(__uint_as_float(x[2 * e + 1]));
                                sum = f2_add(sum, f2_pack(a, b));
                                p[e] = pack16<true>(a, b);
                            }
                            at_st16(pa + j / 2, p);
                        }
                    } else {
                        all = 0.f;
#pragma unroll 1
                        for (int j = 0; j < 64; j += 4) {
                            uint32_t x[4], p[2];
                            at_ld4(sa + j, x);
                            const float4 k4 = ck[j / 4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float a = exponent(x[e], k4, e, base);
                                all += ex2_approx(a);
                                const float w = ex2_approx(a + ve[j + e]);
                                sum = f2_add(sum, f2_pack(w, 0.f));
                                x[e] = __float_as_uint(w);
                            }
                            p[0] = pack16<true>(__uint_as_float(x[0]), __uint_as_float(x[1]));
                            p[1] = pack16<true>(__uint_as_float(x[2]), __uint_as_float(x[3]));
                            at_st2(pa + j / 2, p);
                        }
                    }
                    f2_unpack(sum, s0, s1);
                    if (again || __builtin_expect(!any_of_rows(!(s0 + s1 <= 32768.f && all <= 0x1p107f) || ref == -INFINITY), 1)) break;
                    float mx = -INFINITY;
                    if (__builtin_expect(!wide, 1)) {
#pragma unroll 1
                        for (int j = 0; j < 64; j += 32) {
                            uint32_t x[32];
                            exponents(x, j, base);
#pragma unroll
                            for (int e = 0; e < 32; ++e) mx = fmaxf(mx, __uint_as_float(x[e]));
                        }
                    } else {
#pragma unroll 1
                        for (int j = 0; j < 64; j += 4) {
                            uint32_t x[4];
                            at_ld4(sa + j, x);
                            const float4 k4 = ck[j / 4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                mx = fmaxf(mx, exponent(x[e], k4, e, base) + fmaxf(ve[j + e], AT_LEAST));
                        }
                    }
                    sm_ref[half][r] = mx;
                    sync_rows();  // (the next write is behind the next vote)
                    mx = fmaxf(mx, sm_ref[half ^ 1][r]);
                    const float to = fmaxf(ref, base + ceilf(mx) - AT_TOP);  // whole, so that sums are rescaled exactly
                    const float f = ref == to ? 1.f : exp2_down(to - ref);
                    tot *= f;
                    if (t > s.t0) {  // O holds sums by the old reference
                        wait(&pv[(i - 1) & 1], (i - 1) >> 1);
                        scale_rows<CH>(tbase + lanes + T_O + half * CH, f);
                    }
                    ref = to;
                }
                tot = wide ? tot + all : fmaf(s0 + s1, exp2_int(-unit_i), tot);
                if (__builtin_expect(tail && half == 0, 0)) {
                    const uint32_t bad = clean_values<true, DP>(sm_v + (i & 1) * S::OPERAND, t0, s, tid);
                    if (bad) atomicOr(&bad_nodes[seg & 1], bad);
                    fence_proxy_async_smem();
                }
                at_st_wait();
                at_before();
                __syncwarp();
                if (lane == 0) at_arrive(&pf[i & 1]);
            }
            // the next segment's queries (every product of this one's is done)
            const Segment done = s;
            sm_tot[half][r] = tot;
            sync();  // every warp has marked its nodes
            tot += sm_tot[half ^ 1][r];
            const uint32_t nodes_bad = bad_nodes[seg & 1];
            // the other word is for the next segment, which starts when all
            // eight warps have arrived at qf: nobody reads or marks it now
            if (tid == 0 && half == 0) bad_nodes[(seg & 1) ^ 1] = 0;
            if (more) {
                s = after;
                load_q(s);
            }
            // (the last scores say that all products but the last two are done,
            // so that of either barrier only the last phase can be open)
            wait(&pv[(i - 1) & 1], (i - 1) >> 1);
            at_after();
            put_tile<SPEC_E4M3, DP>(A, share, done, tbase + lanes + T_O, r, node, nodes_bad & mask, ref, tot, half * CH,
                                     half * CH + CH);
            at_before();
            __syncwarp();
            if (lane == 0) at_arrive(&of);
            if (!more) break;
        }
    } else if (warp >= 12) {
        // ---- V to f16: 4 lanes a token, two 16-byte chunks (16 channels each) a
        // lane, 2 tokens a thread.  Eight lanes take tokens t and t ^ 5: their
        // swizzles differ in the top bit, so that reads are from all banks at once,
        // and in the lowest, so that writes are.
        const int tid = threadIdx.x - 384, x = lane & 3, odd = lane >> 2 & 1;
        const int tok0 = (warp - 12) * 8 + ((lane >> 3) ^ (odd * 5));
        uint32_t i = 0;
        int b_at = first;
        for (long long g = share.begin; g < share.end;) {
            const Segment s = segment_at(A, L, share, g, b_at);
            b_at = s.b;
            g = s.g + s.t1 - s.t0;
            for (int t = s.t0; t < s.t1; ++t, ++i) {
                const int valid = s.ctx + s.n - t * 128;
                const uint32_t rs = i % NR, st = i & 1;
                const uint8_t* raw = sm_raw + (rs * 2 + 1) * S::RAW;
                const uint8_t* sc = sm_sc + rs * 256 + 128;
                uint8_t* out = sm_v + st * S::OPERAND;
                wait(&rvf[rs], i / NR);
                // the largest scale byte of the tile's valid tokens, and whether some is far below
                const uint32_t bytes = *reinterpret_cast<const uint32_t*>(sc + lane * 4);
                const int left = valid - lane * 4;
                const uint32_t there = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
                uint32_t z = bytes & there;
                z = __vmaxu4(z, z >> 16);
                const int top = int(__reduce_max_sync(0xffffffffu, max(z & 255u, z >> 8 & 255u)));
                const uint32_t least = uint32_t(max(min(top, 253) - AT_SPREAD, 0)) * 0x01010101u;
                const bool wide = __any_sync(0xffffffffu, __vcmpltu4(bytes, least) & there);
                const int unit = wide ? AT_WIDE : max(min(max(top, 1), 253) - 127, int(AT_LEAST));
                uint4 q[2][2];
                uint32_t f[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int tk = tok0 + k * 64;
                    f[k] = wide ? 0x3c003c00u : half2_exp2(min(min(max(int(sc[tk]), 1), 253) - 127 - unit, 0));
#pragma unroll
                    for (int h = 0; h < S::HALVES; ++h)
                        q[k][h] = *reinterpret_cast<const uint4*>(raw + tk * 128 + (((x + h * 4) ^ (tk & 7)) << 4));
                }
                wait(&ve[st], (i >> 1) ^ 1u);
                if (tid == 0) unit_v[st] = unit;
                if (wide && warp == 13)
                    *reinterpret_cast<float4*>(&sm_ve[st][lane * 4]) =
                        make_float4(float(min(max(int(bytes & 255u), 1), 253) - 127), float(min(max(int(bytes >> 8 & 255u), 1), 253) - 127),
                                    float(min(max(int(bytes >> 16 & 255u), 1), 253) - 127), float(min(max(int(bytes >> 24), 1), 253) - 127));
                if (warp == 12) {  // K's factors, 4 tokens a lane (1 past the request's end)
                    wait(&rkf[rs], i / NR);
                    const uint32_t w = *reinterpret_cast<const uint32_t*>(sm_sc + rs * 256 + lane * 4);
                    float c4[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        c4[e] = e < left ? exp2_int(min(max(int(w >> (8 * e) & 255u), 1), 253) - 127) : 1.f;
                    *reinterpret_cast<float4*>(&sm_ck[st][lane * 4]) = make_float4(c4[0], c4[1], c4[2], c4[3]);
                    __syncwarp();
                    if (lane == 0) at_arrive(&rke[rs]);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int h = 0; h < S::HALVES; ++h) {
                        const int tk = tok0 + k * 64;
                        const uint32_t u[4] = {q[k][h].x, q[k][h].y, q[k][h].z, q[k][h].w};
                        uint32_t v[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            v[2 * e] = half2_mul(e4m3x2_to_f16x2(uint16_t(u[e])), f[k]);
                            v[2 * e + 1] = half2_mul(e4m3x2_to_f16x2(uint16_t(u[e] >> 16)), f[k]);
                        }
                        uint8_t* o = out + h * 16384 + tk * 128;
                        *reinterpret_cast<uint4*>(o + (((2 * x) ^ (tk & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
                        *reinterpret_cast<uint4*>(o + (((2 * x + 1) ^ (tk & 7)) << 4)) = make_uint4(v[4], v[5], v[6], v[7]);
                    }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    at_arrive(&vf[st]);
                    at_arrive(&rve[rs]);
                }
            }
        }
    }

    at_before();
    __syncthreads();
    at_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tbase) : "memory");
    if (threadIdx.x == 0 && *gone && A.status) atomicOr(A.status, int(SPEC_BADBIT_TIMEOUT));
}

template <int DP>
cudaError_t launch_tiles_e4m3(const AttnLaunch& L) {
    using S = TilesE4Shape<DP>;
    static bool ready[64] = {};  // per device; setting it twice does no harm
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev]) {
        e = cudaFuncSetAttribute(k_attn_tiles_e4m3<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(S::SMEM));
        if (e != cudaSuccess) return e;
        ready[dev] = true;
    }
    e = launch_behind(k_attn_tiles_e4m3<DP>, dim3(unsigned(L.ctas)), S::THREADS, S::SMEM, L.st, L.mk, L.mv, L.A);
    return e == cudaSuccess ? launch_attn_join(L, DP) : e;
}

}  // namespace sv
