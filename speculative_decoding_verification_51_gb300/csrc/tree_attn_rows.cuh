// tree_attn_rows.cuh -- k_attn_rows: the attention for few rows a key head
// (16 a tile), where the cache's bytes are what counts: 256 chains of 4 nodes and 4
// query heads a key head over 64 to 4096 tokens of 16 bits take 330 us, 0.99 of the
// measured copy rate; one token over 777 tokens 8.5 us, which is latency.
//
// A CTA (one per SM) has 8 warps, and every warp is a pipeline of its own: it
// takes every eighth chunk of 16 tokens of the segment, loads the chunk's K
// and V rows by TMA into its own ring of stages (a chunk lies in one page,
// whose size is a multiple of 16), and keeps the running reference, total and
// sums of all rows of the tile in its registers.  No warp waits for another
// until the segment ends, when the eight states are joined in shared memory.
//
// Mathematics.  With scores in powers of two, s_t = c q.k_t, and a reference
// m: o = sum_t 2^(s_t - m) v_t / sum_t 2^(s_t - m), for any m.  The reference
// is raised only when a chunk's maximum passes it by 2^6, so that the sums are
// seldom rescaled; the weights stay below 2^6 times the chunk's 16 tokens,
// far inside float32 (the sums) and both 16-bit types (the weights).
//
// Products are mma.sync m16n8k16 on 16-bit operands with float32 sums: with 16
// rows a chunk's 8 KB (128 channels) need 32 of them, a small part of what an SM
// does in the 350 cycles that HBM takes to deliver the chunk.  tcgen05 would pad
// 16 rows to 128.
//
// e4m3 rows.  ldmatrix moves byte pairs, so a lane gets 4 consecutive channels
// of a K row where the 16-bit fragment has two pairs 8 apart; the query's
// channels are permuted alike in shared memory, which leaves the products'
// sum as it is.  V comes transposed in pairs of channels: a byte permutation
// separates even channels from odd, and the accumulator's columns are then
// channels 4 apart.  Both are converted to f16, exactly.  K's scale multiplies
// the score; V's scale 2^e joins the exponent of its weight, w_t = 2^(s_t + e_t -
// m) with m the running maximum of s_t + e_t: then the weights are as large as
// their tokens' contributions, and f16's range is no limit.  The total is the
// sum of 2^(s_t - m).  The reference takes e_t at -100 or more, so that a row
// of zeros (e = -126) does not push the total out of float32.
#pragma once

#include "ring.cuh"
#include "tree_attn.cuh"

namespace sv {

constexpr float AR_SLACK = 6.f;

template <int KIND, int NK>
struct RowsShape {
    static constexpr bool E4 = KIND == SPEC_E4M3;
    static constexpr int DP = NK * 16, R = 16;
    // eight warps, or four where the stages of eight would not fit
    static constexpr int WARPS = !E4 && NK > 8 ? 4 : 8, THREADS = WARPS * 32;
    static constexpr int BOXES = E4 ? (DP + 127) / 128 : (DP + 63) / 64;  // 128 bytes of a row each
    static constexpr int SIDE = BOXES * 2048;                             // K (or V) of a chunk
    static constexpr int STAGE = 2 * SIDE;
    // one warp's sums, at the join: pitches that spread 8 rows over all banks
    static constexpr int OP = E4 ? DP + 16 : DP + 8, OB = R * OP * 4;
    static constexpr int FIXED = 4 * OB + R * (DP + 8) * 2 + (2 * WARPS + 4) * R * 4 + 4096;
    static constexpr int ROOM = (232448 - 1024 - int(sizeof(PlanWindow)) - FIXED) / (WARPS * STAGE);
    static constexpr int STAGES = ROOM < 6 ? ROOM : 6;
    static_assert(STAGES >= 2, "no room for a ring");
    static constexpr size_t SMEM = 1024 + size_t(WARPS) * STAGES * STAGE + FIXED;
    // the query's fragments stay in registers where they are few
    static constexpr bool QREG = NK <= 8;
};

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}
template <bool F16>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, "
            "%7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int KIND, int NK>
__global__ void __launch_bounds__(RowsShape<KIND, NK>::THREADS, 1)
    k_attn_rows(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                const __grid_constant__ AttnArgs A) {
    using S = RowsShape<KIND, NK>;
    constexpr bool E4 = S::E4, F16 = KIND != SPEC_BF16;
    constexpr int DP = S::DP, R = S::R, OP = S::OP, QP = DP + 8, AR_WARPS = S::WARPS, AR_THREADS = S::THREADS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* ring = smem + size_t(warp) * S::STAGES * S::STAGE;
    float* sm_o = reinterpret_cast<float*>(smem + size_t(AR_WARPS) * S::STAGES * S::STAGE);
    uint16_t* sm_q = reinterpret_cast<uint16_t*>(sm_o + 4 * R * OP);
    float* sm_m = reinterpret_cast<float*>(sm_q + R * QP);  // [warps][R]
    float* sm_l = sm_m + AR_WARPS * R;
    float* sm_ref = sm_l + AR_WARPS * R;   // [R] joined reference
    float* sm_tot = sm_ref + R;            // [R] joined total
    uint32_t* sm_qmax = reinterpret_cast<uint32_t*>(sm_tot + R);  // [R]
    uint32_t* sm_mask = sm_qmax + R;                              // [R]
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm_mask + R);    // [warps][stages]
    uint8_t* sm_sc = reinterpret_cast<uint8_t*>(bars + AR_WARPS * S::STAGES);  // [warps][stages][32]
    int* sm_flag = reinterpret_cast<int*>(sm_sc + AR_WARPS * S::STAGES * 32);  // [2]
    uint64_t* bar = bars + warp * S::STAGES;
    uint8_t* sc = sm_sc + warp * S::STAGES * 32;

    __shared__ PlanWindow window;
    if (lane == 0) {
        for (int i = 0; i < S::STAGES; ++i) mbar_init(&bar[i], 1);
        fence_mbarrier_init();
    }
    if (threadIdx.x == 0) sm_flag[1] = 0;
    __syncwarp();
    begin_after_previous();
    Share share;
    if (!read_plan(A, window, share)) return;  // the whole CTA
    const int first = window.b0;
    const Lists L = {window, A.plan, first};

    // ---- a segment's query rows: read while the segment before it is joined
    constexpr int QV = R * DP / 8, QN = (QV + AR_THREADS - 1) / AR_THREADS;  // vectors of 8 channels
    uint4 qn[QN];
    uint32_t mask_n = 0;
    auto fetch = [&](const Segment& s) {
#pragma unroll
        for (int k = 0; k < QN; ++k) {
            const int i = threadIdx.x + k * AR_THREADS, r = i / (DP / 8), d = (i - r * (DP / 8)) * 8, row = s.rt * R + r;
            const int v = row / A.G;
            qn[k] = make_uint4(0, 0, 0, 0);
            if (i < QV && row < A.rows && d < A.D && v < s.n)
                qn[k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(A.q) + s.b * A.qb + v * A.qn +
                                                             (s.h * A.G + row - v * A.G) * A.qh + d));
        }
        const int row = s.rt * R + int(threadIdx.x), v = row / A.G;
        mask_n = 0;
        if (threadIdx.x < R && row < A.rows && v < s.n)
            mask_n = __ldg(A.masks + (long long)s.b * A.N + v) & (0xffffffffu >> (32 - s.n));
    };

    const Segment ps0 = segment_at(A, L, share, share.begin, first);
    fetch(ps0);  // before the copies, which would hold it up

    // ---- this warp's copies.  Lane l holds the page of the l-th next chunk of the
    // warp (one read every 32 chunks: read one by one, each would wait for L2 or
    // HBM before its copies could start).
    Segment ps = ps0;
    int pc = ps.c0 + warp, page_at = 0, off_at = 0, pages = 0, ahead = 0;
    bool more = true;
    auto seek = [&]() {  // to the next chunk this warp has, if any
        while (pc >= ps.c1) {
            const long long g = ps.g + (ps.t1 - ps.t0);
            if (g >= share.end) {
                more = false;
                return;
            }
            ps = segment_at(A, L, share, g, ps.b);
            pc = ps.c0 + warp;
            ahead = 0;
        }
        if ((ahead & 31) == 0) {
            const int c = pc + lane * AR_WARPS;
            pages = c < ps.c1 ? __ldg(A.table + (long long)ps.b * A.max_pages + c * 16 / A.page) : 0;
        }
        page_at = page_in(A, __shfl_sync(0xffffffffu, pages, ahead & 31));
        ++ahead;
        off_at = pc * 16 % A.page;
    };
    seek();
    CopyRing<S::STAGES> copies;
    auto issue = [&]() {
        if (!more || !copies.alive()) return;
        const uint32_t st = copies.begin();
        if (lane == 0) {
            uint8_t* d = ring + st * S::STAGE;
            mbar_arrive_expect_tx(&bar[st], uint32_t(S::STAGE) + (E4 ? 32u : 0u));
#pragma unroll
            for (int x = 0; x < S::BOXES; ++x) {
                tma_load_4d(d + x * 2048, &mk, x * (E4 ? 128 : 64), off_at, ps.h, page_at, &bar[st]);
                tma_load_4d(d + S::SIDE + x * 2048, &mv, x * (E4 ? 128 : 64), off_at, ps.h, page_at,
                            &bar[st]);
            }
            if constexpr (E4) {
                const long long at = ((long long)page_at * A.Hkv + ps.h) * A.page + off_at;
                bulk_g2s(sc + st * 32, A.ks + at, 16, &bar[st]);
                bulk_g2s(sc + st * 32 + 16, A.vs + at, 16, &bar[st]);
            }
        }
        pc += AR_WARPS;
        seek();
    };
    for (int i = 0; i < S::STAGES; ++i) issue();

    Segment s = ps0;
    for (;;) {
        // ---- the query's rows to shared memory (e4m3: as f16, a power of two
        // a row bringing its largest value to [1, 2))
        if constexpr (E4) {
            for (int r = threadIdx.x; r < R; r += AR_THREADS) sm_qmax[r] = 0;
            __syncthreads();
            auto pair = [&](uint32_t u) {
                return A.q_f16 ? __half22float2(*reinterpret_cast<const __half2*>(&u)) : make_float2(bf16_lo(u), bf16_hi(u));
            };
#pragma unroll
            for (int k = 0; k < QN; ++k) {
                const int i = threadIdx.x + k * AR_THREADS;
                const uint32_t u[4] = {qn[k].x, qn[k].y, qn[k].z, qn[k].w};
                float m = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = pair(u[e]);
                    m = fmaxf(m, fmaxf(finite_abs(f.x), finite_abs(f.y)));
                }
                if (i < QV) atomicMax(&sm_qmax[i / (DP / 8)], __float_as_uint(m));
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < QN; ++k) {
                const int i = threadIdx.x + k * AR_THREADS, r = i / (DP / 8), d = (i - r * (DP / 8)) * 8;
                if (i >= QV) break;
                const uint32_t u[4] = {qn[k].x, qn[k].y, qn[k].z, qn[k].w};
                // 2^-e for the row's exponent e (its largest value >= 2^-126)
                const uint32_t ex = max(min(sm_qmax[r] >> 23, 253u), 1u);
                const float f2 = __uint_as_float((254u - ex) << 23);
                uint32_t h[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = pair(u[e]);
                    h[e] = pack16<true>(f.x * f2, f.y * f2);
                }
                // channels d = 16 j + 4 t + e of a lane's K fragment go to
                // 2 t + e (e < 2) and 8 + 2 t + e - 2
                uint32_t* dst = reinterpret_cast<uint32_t*>(sm_q + r * QP + (d & ~15) + ((d & 8) ? 4 : 0));
                dst[0] = h[0];
                dst[1] = h[2];
                dst[4] = h[1];
                dst[5] = h[3];
            }
        } else {
#pragma unroll
            for (int k = 0; k < QN; ++k) {
                const int i = threadIdx.x + k * AR_THREADS, r = i / (DP / 8), d = (i - r * (DP / 8)) * 8;
                if (i < QV) *reinterpret_cast<uint4*>(sm_q + r * QP + d) = qn[k];
            }
        }
        if (threadIdx.x < R) sm_mask[threadIdx.x] = mask_n;
        __syncthreads();

        // ---- this warp's chunks
        const uint32_t qa = smem_u32(sm_q) + (((lane & 7) + ((lane >> 3) & 1) * 8) * QP + (lane >> 4) * 8) * 2;
        uint32_t qf[S::QREG ? NK : 1][4];
        if constexpr (S::QREG) {
#pragma unroll
            for (int k = 0; k < NK; ++k) ldsm4(qa + k * 32, qf[k]);
        }
        float o[2 * NK][4], ref[2], tot[2], rc[2];
        uint32_t mask[2];
#pragma unroll
        for (int n = 0; n < 2 * NK; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int r = x * 8 + (lane >> 2);
            ref[x] = -INFINITY;
            tot[x] = 0.f;
            mask[x] = sm_mask[r];
            rc[x] = A.c;
            if constexpr (E4) rc[x] = A.c * exp2_int(int(max(min(sm_qmax[r] >> 23, 253u), 1u)) - 127);
        }
        uint32_t v_bad = 0;  // nodes of which some value is not finite
        for (int c = s.c0 + warp; c < s.c1; c += AR_WARPS) {
            const uint32_t st = copies.stage();
            uint8_t* kp = ring + st * S::STAGE;
            uint8_t* vp = kp + S::SIDE;
            // (where a copy did not arrive in time: no more copies and waits)
            if (copies.alive() && __any_sync(0xffffffffu, !mbar_wait_bounded(&bar[st], copies.parity()))) {
                copies.lose();
                if (lane == 0 && A.status) atomicOr(A.status, int(SPEC_BADBIT_TIMEOUT));
            }
            copies.next();
            const int t0 = c * 16;
            const bool tail = t0 + 16 > s.ctx;

            // scores
            float p[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) p[n][e] = 0.f;
            const uint32_t ka = smem_u32(kp);
            if constexpr (E4) {
                const int tk = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
                for (int k = 0; k < NK; k += 2) {
                    uint32_t w[4];
                    const int j = k + (lane >> 4);
                    ldsm4(ka + (j >> 3) * 2048 + tk * 128 + (((j & 7) ^ (tk & 7)) << 4), w);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t b00 = e4m3x2_to_f16x2(uint16_t(w[2 * i])),
                                       b01 = e4m3x2_to_f16x2(uint16_t(w[2 * i] >> 16)),
                                       b10 = e4m3x2_to_f16x2(uint16_t(w[2 * i + 1])),
                                       b11 = e4m3x2_to_f16x2(uint16_t(w[2 * i + 1] >> 16));
                        uint32_t a[4];
                        if constexpr (S::QREG) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) a[e] = qf[k + i][e];
                        } else {
                            ldsm4(qa + (k + i) * 32, a);
                        }
                        mma16<true>(p[0], a, b00, b01);
                        mma16<true>(p[1], a, b10, b11);
                    }
                }
            } else {
                const int tk = (lane & 7) + (lane >> 4) * 8;
#pragma unroll
                for (int k = 0; k < NK; ++k) {
                    uint32_t w[4];
                    const int j = 2 * k + ((lane >> 3) & 1);
                    ldsm4(ka + (j >> 3) * 2048 + tk * 128 + (((j & 7) ^ (tk & 7)) << 4), w);
                    uint32_t a[4];
                    if constexpr (S::QREG) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) a[e] = qf[k][e];
                    } else {
                        ldsm4(qa + k * 32, a);
                    }
                    mma16<F16>(p[0], a, w[0], w[1]);
                    mma16<F16>(p[1], a, w[2], w[3]);
                }
            }
            // this lane's tokens: t0 + 8 n + 2 (lane % 4) + e
            float kf[2][2], ve[2][2];
            if constexpr (E4) {
                const uint8_t* z = sc + st * 32;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const uint16_t a = *reinterpret_cast<const uint16_t*>(z + n * 8 + 2 * (lane & 3));
                    const uint16_t b = *reinterpret_cast<const uint16_t*>(z + 16 + n * 8 + 2 * (lane & 3));
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        kf[n][e] = exp2_int(min(max(int((a >> (8 * e)) & 255), 1), 253) - 127);
                        ve[n][e] = float(min(max(int((b >> (8 * e)) & 255), 1), 253) - 127);
                    }
                }
            }
            bool raise = false;
            float top[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                top[x] = -INFINITY;
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float v = p[n][2 * x + e] * rc[x];
                        if constexpr (E4) v *= kf[n][e];
                        if (tail) {
                            const int u = t0 + n * 8 + 2 * (lane & 3) + e - s.ctx;
                            if (u >= 0 && (u >= 32 || !(mask[x] >> u & 1u))) v = -INFINITY;
                        }
                        p[n][2 * x + e] = v;
                        if constexpr (E4) v += fmaxf(ve[n][e], -100.f);
                        top[x] = fmaxf(top[x], v);
                    }
                top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 1));
                top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 2));
                raise |= top[x] > ref[x] + AR_SLACK;
            }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float to = top[x] > ref[x] + AR_SLACK ? top[x] : ref[x];
                    // a reference of -inf has sums of zero
                    const float f = ref[x] == to ? 1.f : ex2_approx(ref[x] - to);
                    ref[x] = to;
                    tot[x] *= f;
#pragma unroll
                    for (int n = 0; n < 2 * NK; ++n) {
                        o[n][2 * x] *= f;
                        o[n][2 * x + 1] *= f;
                    }
                }
            }
            // weights
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float at = ref[x] == -INFINITY ? 0.f : ref[x];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float v = p[n][2 * x + e] - at;
                        if constexpr (E4) {
                            tot[x] += ex2_approx(v);
                            v = ex2_approx(v + ve[n][e]);
                        } else {
                            v = ex2_approx(v);
                            tot[x] += v;
                        }
                        p[n][2 * x + e] = v;
                    }
            }
            // values of tokens past the request's end, and values of nodes
            // that are not finite, must not meet a weight of zero
            if (tail) {
                uint32_t bad = 0;
                for (int i = lane; i < S::SIDE / 16; i += 32) {
                    const int t = t0 + ((i & 127) >> 3);
                    if (t < s.ctx) continue;
                    uint4* w = reinterpret_cast<uint4*>(vp) + i;
                    if (t >= s.ctx + s.n) {
                        *w = make_uint4(0, 0, 0, 0);
                        continue;
                    }
                    uint32_t u[4] = {w->x, w->y, w->z, w->w};
                    bool hit = false;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if constexpr (E4) {
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                if ((u[e] >> (8 * y) & 0x7fu) == 0x7fu) {
                                    u[e] &= ~(0xffu << (8 * y));
                                    hit = true;
                                }
                        } else {
                            constexpr uint32_t EX = F16 ? 0x7c00u : 0x7f80u;
#pragma unroll
                            for (int y = 0; y < 2; ++y)
                                if ((u[e] >> (16 * y) & EX) == EX) {
                                    u[e] &= ~(0xffffu << (16 * y));
                                    hit = true;
                                }
                        }
                    }
                    if (hit) {
                        *w = make_uint4(u[0], u[1], u[2], u[3]);
                        bad |= 1u << (t - s.ctx);
                    }
                }
                v_bad |= __reduce_or_sync(0xffffffffu, bad);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the stage's next copy
                __syncwarp();
            }
            // sums
            const uint32_t va = smem_u32(vp);
            uint32_t a[4];
            a[0] = pack16<F16>(p[0][0], p[0][1]);
            a[1] = pack16<F16>(p[0][2], p[0][3]);
            a[2] = pack16<F16>(p[1][0], p[1][1]);
            a[3] = pack16<F16>(p[1][2], p[1][3]);
            const int tv = (lane & 7) + ((lane >> 3) & 1) * 8;
            if constexpr (E4) {
#pragma unroll
                for (int k = 0; k < NK; k += 2) {
                    uint32_t w[4];
                    const int j = k + (lane >> 4);
                    ldsm4t(va + (j >> 3) * 2048 + tv * 128 + (((j & 7) ^ (tv & 7)) << 4), w);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t lo = __byte_perm(w[2 * i], 0, 0x3120),
                                       hi = __byte_perm(w[2 * i + 1], 0, 0x3120);
                        const uint32_t e0 = e4m3x2_to_f16x2(uint16_t(lo)),
                                       o0 = e4m3x2_to_f16x2(uint16_t(lo >> 16)),
                                       e1 = e4m3x2_to_f16x2(uint16_t(hi)),
                                       o1 = e4m3x2_to_f16x2(uint16_t(hi >> 16));
                        mma16<true>(o[2 * (k + i)], a, e0, e1);
                        mma16<true>(o[2 * (k + i) + 1], a, o0, o1);
                    }
                }
            } else {
#pragma unroll
                for (int k = 0; k < NK; ++k) {
                    uint32_t w[4];
                    const int j = 2 * k + (lane >> 4);
                    ldsm4t(va + (j >> 3) * 2048 + tv * 128 + (((j & 7) ^ (tv & 7)) << 4), w);
                    mma16<F16>(o[2 * k], a, w[0], w[1]);
                    mma16<F16>(o[2 * k + 1], a, w[2], w[3]);
                }
            }
            __syncwarp();  // every lane is done with the stage
            issue();
        }

        const long long next = s.g + (s.t1 - s.t0);
        Segment after = s;
        if (next < share.end) {
            after = segment_at(A, L, share, next, s.b);
            fetch(after);
        }

        // ---- join the warps
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float l = tot[x];
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            if ((lane & 3) == 0) {
                const int r = x * 8 + (lane >> 2);
                sm_m[warp * R + r] = ref[x];
                sm_l[warp * R + r] = l;
            }
        }
        if (lane == 0 && v_bad) atomicOr(reinterpret_cast<unsigned*>(&sm_flag[1]), v_bad);
        __syncthreads();
        if (threadIdx.x < R) {
            float mm = -INFINITY, l = 0.f;
#pragma unroll
            for (int w = 0; w < AR_WARPS; ++w) mm = fmaxf(mm, sm_m[w * R + threadIdx.x]);
            const float at = mm == -INFINITY ? 0.f : mm;
#pragma unroll
            for (int w = 0; w < AR_WARPS; ++w)
                l += sm_l[w * R + threadIdx.x] * ex2_approx(sm_m[w * R + threadIdx.x] - at);
            sm_ref[threadIdx.x] = mm;
            sm_tot[threadIdx.x] = l;
        }
        float* ob = sm_o + (warp & 3) * R * OP;
#pragma unroll
        for (int half = AR_WARPS / 4 - 1; half >= 0; --half) {
            if ((warp >> 2) == half) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int r = x * 8 + (lane >> 2);
                    float mm = -INFINITY;
#pragma unroll
                    for (int w = 0; w < AR_WARPS; ++w) mm = fmaxf(mm, sm_m[w * R + r]);
                    const float f = ref[x] == -INFINITY ? 0.f : ex2_approx(ref[x] - mm);
                    float* z = ob + r * OP;
                    const bool first_half = half == AR_WARPS / 4 - 1;
                    if constexpr (E4) {  // accumulators 2 j and 2 j + 1: channels 16 j + 4 t + {0, 2}, {1, 3}
#pragma unroll
                        for (int j = 0; j < NK; ++j) {
                            float4* y = reinterpret_cast<float4*>(z + j * 16 + 4 * (lane & 3));
                            float4 v = make_float4(o[2 * j][2 * x] * f, o[2 * j + 1][2 * x] * f,
                                                   o[2 * j][2 * x + 1] * f, o[2 * j + 1][2 * x + 1] * f);
                            if (!first_half) {
                                const float4 b = *y;
                                v = make_float4(v.x + b.x, v.y + b.y, v.z + b.z, v.w + b.w);
                            }
                            *y = v;
                        }
                    } else {
#pragma unroll
                        for (int n = 0; n < 2 * NK; ++n) {
                            float2* y = reinterpret_cast<float2*>(z + n * 8 + 2 * (lane & 3));
                            float2 v = make_float2(o[n][2 * x] * f, o[n][2 * x + 1] * f);
                            if (!first_half) {
                                const float2 b = *y;
                                v = make_float2(v.x + b.x, v.y + b.y);
                            }
                            *y = v;
                        }
                    }
                }
            }
            __syncthreads();
        }
        const bool whole = s.t0 == 0 && s.t1 == s.tiles;
        const uint32_t bad_nodes = uint32_t(sm_flag[1]);
        const long long slot = part_slot(share, s);
        for (int i = threadIdx.x; i < R * (DP / 4); i += AR_THREADS) {
            // a whole item: channels side by side, as in the output; a part: rows
            // side by side, as in the workspace
            const int r = whole ? i / (DP / 4) : i % R, d = (whole ? i - r * (DP / 4) : i / R) * 4;
            const int row = s.rt * R + r;
            if (row >= A.rows) continue;
            float4 x = *reinterpret_cast<const float4*>(sm_o + r * OP + d);
#pragma unroll
            for (int w = 1; w < 4; ++w) {
                const float4 y = *reinterpret_cast<const float4*>(sm_o + w * R * OP + r * OP + d);
                x.x += y.x;
                x.y += y.y;
                x.z += y.z;
                x.w += y.w;
            }
            float v[4] = {x.x, x.y, x.z, x.w};
            if (bad_nodes & sm_mask[r])  // values that are not finite, for the rows that see them
                for (uint32_t m = bad_nodes & sm_mask[r]; m; m &= m - 1)
                    for (int e = 0; e < 4; ++e)
                        if (d + e < A.D) v[e] += not_finite_v<KIND>(A, s.b, s.h, s.ctx + __ffs(m) - 1, d + e);
            if (whole) {
                put_row(A, s, row, d, v, sm_tot[r]);
                if (d == 0) put_lse(A, s, row, sm_ref[r], sm_tot[r]);
            } else {
                reinterpret_cast<float4*>(A.part_o)[(slot * (DP / 4) + d / 4) * R + r] = make_float4(v[0], v[1], v[2], v[3]);
                if (d == 0)
                    *reinterpret_cast<float2*>(A.part_ml + (slot * R + r) * 2) = make_float2(sm_ref[r], sm_tot[r]);
            }
        }
        if (!whole) join_parts<2>(A, share, s, R, DP, sm_flag, threadIdx.x, AR_THREADS, 0);
        __syncthreads();
        if (next >= share.end) break;
        if (threadIdx.x == 0) sm_flag[1] = 0;
        s = after;
    }
    copies.drain([&](uint32_t st, uint32_t parity) { mbar_wait_bounded(&bar[st], parity, 100000000ull); });
}

template <int KIND, int NK>
cudaError_t launch_rows(const AttnLaunch& L) {
    using S = RowsShape<KIND, NK>;
    static bool ready[64] = {};  // per device; setting it twice does no harm
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev]) {
        e = cudaFuncSetAttribute(k_attn_rows<KIND, NK>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(S::SMEM));
        if (e != cudaSuccess) return e;
        ready[dev] = true;
    }
    return launch_behind(k_attn_rows<KIND, NK>, dim3(unsigned(L.ctas)), S::THREADS, S::SMEM, L.st, L.mk, L.mv, L.A);
}

template <int KIND>
cudaError_t launch_rows_any(const AttnLaunch& L) {
    const int D = L.A.D;
    return D <= 64    ? launch_rows<KIND, 4>(L)
           : D <= 96  ? launch_rows<KIND, 6>(L)
           : D <= 128 ? launch_rows<KIND, 8>(L)
                      : launch_rows<KIND, 16>(L);
}

}  // namespace sv
