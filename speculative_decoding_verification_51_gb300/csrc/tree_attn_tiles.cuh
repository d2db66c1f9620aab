// tree_attn_tiles.cuh -- k_attn_tiles: the attention for many rows a key head
// (up to 128 a tile) over a 16-bit cache, on the tcgen05 tensor cores.
//
// One CTA per SM, warps by role:
//   warp 0        TMA: the K and V rows of a tile of 128 tokens by the page table,
//                 in boxes as long as a page allows, 128-byte swizzle
//   warp 1        one thread issues the products: S = Q K^T (M = 128 rows, N = 128
//                 tokens) into one of two TMEM buffers, O += P V with P in TMEM
//                 and V as it lies (token rows: a transposed B operand)
//   warps 4..7    softmax, one row a thread: S from TMEM, the weights back to it
//                 as 16-bit P, the row's reference and total in registers;
//                 between segments the next rows of Q, and the finished rows of O
// S of tile i + 1 is computed while the weights of tile i are made.
//
// Two requests of 9 nodes and 8 query heads a key head over 131 K tokens take 167 us:
// 0.95 of the measured copy rate, a quarter of the tensor rate.
//
// As in k_attn_rows the reference of a row is raised only when a score passes
// it by some octaves, so that O in TMEM is seldom rescaled; a weight is then at most
// 2^8 (bf16) or 2^15 (f16), which the types hold and whose rounding is relative.  f16
// ends at 2^-24, and a long context can have much of its weight in a flat tail below: so
// a raised reference leaves the largest f16 weight at 2^8, and the tail counts down to
// 2^-33 of it.
//
// The loops over a tile's columns are rolled where they can be: the roles' code
// together has to stay in the SM's instruction cache.  (Unrolled, the stall
// for instructions was the largest of all, and a tile of an 8-bit cache took
// three times as long.)
#pragma once

#include "tensor.cuh"
#include "tree_attn.cuh"

namespace sv {

template <int DP>
struct TilesShape {
    static constexpr int HALVES = DP / 64;
    static constexpr int OPERAND = HALVES * 16384;  // 128 tokens (or rows) of 16-bit channels
    static constexpr int STAGES = DP == 64 ? 6 : 3;
    static constexpr size_t SMEM = 1024 + size_t(OPERAND) * (1 + 2 * STAGES);
    static_assert(SMEM + 1024 <= 232448, "shared memory");
    static constexpr int THREADS = 256;
};

// `tokens` columns of S in place: what the row does not see becomes -inf.  u0: node
// index of the first one's token (negative: within the context).
__device__ __forceinline__ void hide_unseen(uint32_t sa, int u0, uint32_t mask, int tokens) {
#pragma unroll 1
    for (int j = 0; j < tokens; j += 32) {
        const int u = u0 + j;
        const uint32_t on = u <= -32 ? 0xffffffffu
                            : u < 0  ? (0xffffffffu >> (32 + u)) | (mask << -u)
                            : u < 32 ? mask >> u
                                     : 0u;
        uint32_t f[32], x[16], y[16];
        at_ld32(sa + j, f);
        at_ld_wait(f);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            x[e] = on >> e & 1u ? f[e] : 0xff800000u;
            y[e] = on >> (e + 16) & 1u ? f[e + 16] : 0xff800000u;
        }
        at_st16(sa + j, x);
        at_st16(sa + j + 16, y);
    }
    at_st_wait();
}

// In a tile of values (128 threads): rows past the request's end become zero,
// and so do elements of nodes that are not finite, since neither must meet a
// weight of zero.  Returns the nodes that had such elements.
template <bool F16, int DP>
__device__ __forceinline__ uint32_t clean_values(uint8_t* tile, int t0, const Segment& s, int tid) {
    uint32_t bad = 0;
    for (int x = tid; x < DP * 16; x += 128) {
        const int tok = t0 + ((x >> 3) & 127);
        if (tok < s.ctx) continue;
        uint4* p = reinterpret_cast<uint4*>(tile) + x;
        if (tok >= s.ctx + s.n) {
            *p = make_uint4(0, 0, 0, 0);
            continue;
        }
        uint32_t u[4] = {p->x, p->y, p->z, p->w};
        bool hit = false;
        constexpr uint32_t EX = F16 ? 0x7c00u : 0x7f80u;
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int y = 0; y < 2; ++y)
                if ((u[e] >> (16 * y) & EX) == EX) {
                    u[e] &= ~(0xffffu << (16 * y));
                    hit = true;
                }
        if (hit) {
            *p = make_uint4(u[0], u[1], u[2], u[3]);
            bad |= 1u << (tok - s.ctx);
        }
    }
    return bad;
}

// Channels [from, to) of a thread's finished row (r of the tile; its sums in TMEM
// at o): to the output where the segment is the whole item, else to the workspace.  `bad`: the
// nodes it sees that have values which are not finite.
template <int KIND, int DP>
__device__ __forceinline__ void put_tile(const AttnArgs& A, const Share& share, const Segment& s, uint32_t o,
                                         int r, int node, uint32_t bad, float ref, float tot, int from,
                                         int to) {
    const bool whole = s.t0 == 0 && s.t1 == s.tiles;
    const long long slot = part_slot(share, s);
    const int row = s.rt * 128 + r;
    const bool none = node >= s.n || tot == 0.f;  // as in put_row
    const float inv = none ? 0.f : 1.f / tot;
    const long long at = (((long long)s.b * A.N + node) * A.Hq + s.h * A.G + row - node * A.G) * A.D;
#pragma unroll 1
    for (int j = from; j < to; j += 32) {
        uint32_t u0[32];
        at_ld32(o + j, u0);
        at_ld_wait(u0);
        float f[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(u0[e]);
        if (row < A.rows) {
            for (uint32_t m = bad; m; m &= m - 1)
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (j + e < A.D) f[e] += not_finite_v<KIND>(A, s.b, s.h, s.ctx + __ffs(m) - 1, j + e);
            if (whole) {
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    uint32_t u[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const float lo = none ? 0.f : f[e + 2 * x] * inv, hi = none ? 0.f : f[e + 2 * x + 1] * inv;
                        u[x] = A.q_f16 ? pack16<true>(lo, hi) : pack16<false>(lo, hi);
                    }
                    if (j + e < A.D)
                        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(A.out) + at + j + e) = make_uint4(u[0], u[1], u[2], u[3]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    reinterpret_cast<float4*>(A.part_o)[(slot * (DP / 4) + (j + e) / 4) * 128 + r] = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
            }
        }
        __syncwarp();
    }
    if (from) return;
    if (whole) put_lse(A, s, row, ref, tot);
    else if (row < A.rows) *reinterpret_cast<float2*>(A.part_ml + (slot * 128 + r) * 2) = make_float2(ref, tot);
}

template <int KIND, int DP>
__global__ void __launch_bounds__(TilesShape<DP>::THREADS, 1)
    k_attn_tiles(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                 const __grid_constant__ AttnArgs A) {
    using S = TilesShape<DP>;
    constexpr bool F16 = KIND == SPEC_F16;
    constexpr int ST = S::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    uint8_t* sm_q = smem;
    uint8_t* sm_k = sm_q + S::OPERAND;
    uint8_t* sm_v = sm_k + ST * S::OPERAND;
    __shared__ __align__(8) uint64_t kf[ST], ke[ST], vf[ST], ve[ST];  // stages full and empty
    __shared__ __align__(8) uint64_t sf[2], pf[2], pv[2], qf, of, fin;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    __shared__ uint32_t bad_nodes[2];
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
        for (int i = 0; i < ST; ++i) {
            mbar_init(&kf[i], 1);
            mbar_init(&ke[i], 1);
            mbar_init(&vf[i], 1);
            mbar_init(&ve[i], 1);
        }
        mbar_init(&sf[0], 1);
        mbar_init(&sf[1], 1);
        mbar_init(&pf[0], 4);
        mbar_init(&pf[1], 4);
        mbar_init(&pv[0], 1);
        mbar_init(&pv[1], 1);
        mbar_init(&qf, 4);
        mbar_init(&of, 4);
        mbar_init(&fin, 1);
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
    constexpr uint32_t T_O = 256, T_P = 384;  // S buffers at 0 and 128, then O, and P (64 columns each)
    volatile int* gone = &abort_flag;
    // a bounded wait; once one has run out nobody waits any more
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity & 1u) || *gone) return;
        if (!at_wait_bounded(bar, parity & 1u, AT_WAIT_NS)) *gone = 1;
    };

    if (warp == 0) {
        // ---- copies (K and V from one warp: in turn they keep HBM's pages better; two
        // contexts of 131 K tokens 173 us, with a warp each 178): lane = (128-byte part of
        // the rows, box of A.box tokens)
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
                const uint32_t st = i % ST, ph = i / ST;
                const int in = page_in(A, page);
#pragma unroll
                for (int side = 0; side < 2; ++side) {
                    uint64_t* full = side ? &vf[st] : &kf[st];
                    if (lane == 0) {
                        wait(side ? &ve[st] : &ke[st], ph ^ 1u);
                        if (!*gone) mbar_arrive_expect_tx(full, nv * S::HALVES * box_bytes);
                    }
                    __syncwarp();
                    if (part < S::HALVES && off >= 0 && !*gone)
                        tma_load_4d((side ? sm_v : sm_k) + st * S::OPERAND + part * 16384 + chunk * box_bytes,
                                    side ? &mv : &mk, part * 64, off, s.h, in, full);
                }
                page = page2;
                off = off2;
            }
        }
        // every copy has landed before the CTA leaves (they have, unless a wait ran out)
        if (lane == 0 && *gone) {
            for (uint32_t j = i > ST ? i - ST : 0; j < i; ++j) {
                at_wait_bounded(&kf[j % ST], (j / ST) & 1u, AT_WAIT_NS / 8);
                at_wait_bounded(&vf[j % ST], (j / ST) & 1u, AT_WAIT_NS / 8);
            }
        }
    } else if (warp == 1) {
        // ---- products
        if (lane == 0) {
            constexpr uint32_t id_s = at_idesc<F16>(128, false), id_o = at_idesc<F16>(DP, true);
            uint32_t i = 0, seg = 0;
            int b_at = first;
            const uint32_t qa = smem_u32(sm_q);
            auto scores = [&](uint32_t j) {
                const uint32_t st = j % ST;
                wait(&kf[st], j / ST);
                at_after();
                const uint32_t ka = smem_u32(sm_k) + st * S::OPERAND;
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
                    at_mma_ss(tbase + (j & 1) * 128, at_desc_k(qa + (k >> 2) * 16384 + (k & 3) * 32),
                              at_desc_k(ka + (k >> 2) * 16384 + (k & 3) * 32), id_s, k > 0);
                at_commit(&ke[st]);
                at_commit(&sf[j & 1]);
            };
            for (long long g = share.begin; g < share.end; ++seg) {
                const Segment s = segment_at(A, L, share, g, b_at);
                b_at = s.b;
                g = s.g + s.t1 - s.t0;
                wait(&qf, seg);
                at_after();
                scores(i);
                for (int t = s.t0; t < s.t1; ++t, ++i) {
                    if (t + 1 < s.t1) scores(i + 1);
                    const uint32_t st = i % ST;
                    wait(&vf[st], i / ST);
                    wait(&pf[i & 1], i >> 1);
                    if (t == s.t0) wait(&of, seg ^ 1u);  // the last segment's rows have been read
                    at_after();
                    const uint32_t va = smem_u32(sm_v) + st * S::OPERAND;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        at_mma_ts(tbase + T_O, tbase + T_P + (i & 1) * 64 + k * 8, at_desc_mn(va + k * 2048), id_o,
                                  t > s.t0 || k > 0);
                    at_commit(&ve[st]);
                    at_commit(&pv[i & 1]);
                }
            }
            at_commit(&fin);  // every product is done before TMEM is freed
            at_wait_bounded(&fin, 0, AT_WAIT_NS);
        }
    } else if (warp >= 4 && warp < 8) {
        // ---- softmax: row = this thread's TMEM lane
        const int w = warp - 4, r = w * 32 + lane, tid = r;
        const uint32_t lanes = uint32_t(w * 32) << 16;
        // a factor of zero would make NaN of -inf; no score of this size counts
        const float c = fmaxf(fabsf(A.c), 1e-30f);
        const uint32_t flip = A.c < 0.f ? 0x80008000u : 0u;
        auto sync = [&]() { asm volatile("bar.sync 1, 128;" ::: "memory"); };
        auto load_q = [&](const Segment& s) {
            const int row = s.rt * 128 + r, v = row / A.G;
            const bool on = row < A.rows && v < s.n;
            const uint16_t* src = static_cast<const uint16_t*>(A.q) + s.b * A.qb + v * A.qn +
                                  (s.h * A.G + row - v * A.G) * A.qh;
            uint4 u[DP / 8];  // every load in flight at once
#pragma unroll
            for (int j = 0; j < DP / 8; ++j)
                u[j] = on && j * 8 < A.D ? __ldg(reinterpret_cast<const uint4*>(src + j * 8)) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < DP / 8; ++j)
                *reinterpret_cast<uint4*>(sm_q + (j >> 3) * 16384 + r * 128 + (((j & 7) ^ (r & 7)) << 4)) =
                    make_uint4(u[j].x ^ flip, u[j].y ^ flip, u[j].z ^ flip, u[j].w ^ flip);
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
                const uint32_t sa = tbase + lanes + (i & 1) * 128;
                const uint32_t pa = tbase + lanes + T_P + (i & 1) * 64;  // PV of tile i - 2 is done with it
                const int t0 = t * 128;
                const bool tail = t0 + 128 > s.ctx;
                wait(&sf[i & 1], i >> 1);
                at_after();
                if (__builtin_expect(tail, 0)) hide_unseen(sa, t0 - s.ctx, mask, 128);
                // One pass makes the weights by the reference as it is and finds the
                // largest score; where some row's passes the reference by too
                // much (seldom, but for a segment's first tile), the reference is
                // raised and the weights are made again.
                float s0, s1;
                for (;;) {
                    const float at = ref == -INFINITY ? 0.f : -ref;
                    const uint64_t c2 = f2_pack(c, c), at2 = f2_pack(at, at);
                    uint64_t sum = f2_pack(0.f, 0.f);
                    float mx = -INFINITY;
                    auto piece = [&](const uint32_t (&f)[32], int j) {
                        uint32_t p[16];
                        float m2 = -INFINITY;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float x = __uint_as_float(f[2 * e]), y = __uint_as_float(f[2 * e + 1]);
                            float a, b;
                            m2 = fmaxf(fmaxf(x, y), m2);
                            f2_unpack(f2_fma(f2_pack(x, y), c2, at2), a, b);
                            a = ex2_approx(a);
                            b = ex2_approx(b);
                            sum = f2_add(sum, f2_pack(a, b));
                            p[e] = pack16<F16>(a, b);
                        }
                        mx = fmaxf(mx, m2);
                        at_st16(pa + j / 2, p);
                    };
                    uint32_t f[32], g[32];
                    at_ld32(sa, f);
#pragma unroll 1
                    for (int j = 0; j < 128; j += 64) {
                        at_ld_wait(f);
                        at_ld32(sa + j + 32, g);
                        piece(f, j);
                        at_ld_wait(g);
                        if (j == 0) at_ld32(sa + 64, f);
                        piece(g, j + 32);
                    }
                    f2_unpack(sum, s0, s1);
                    const float top = mx * c;
                    const bool raise = top > ref + TilesRange<F16>::SLACK;
                    if (__builtin_expect(!__any_sync(0xffffffffu, raise), 1)) break;
                    const float to = raise ? top - TilesRange<F16>::TOP : ref;
                    const float f2 = ref == to ? 1.f : ex2_approx(ref - to);
                    ref = to;
                    tot *= f2;
                    if (t > s.t0) {  // O holds sums by the old reference
                        wait(&pv[(i - 1) & 1], (i - 1) >> 1);
                        scale_rows<DP>(tbase + lanes + T_O, f2);
                    }
                }
                tot += s0 + s1;
                if (__builtin_expect(tail, 0)) {
                    const uint32_t st = i % ST;
                    wait(&vf[st], i / ST);
                    const uint32_t bad = clean_values<F16, DP>(sm_v + st * S::OPERAND, t0, s, tid);
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
            sync();  // every warp has marked its nodes
            const uint32_t nodes_bad = bad_nodes[seg & 1];
            // the other word is for the next segment, which starts when all
            // four warps have arrived at qf: nobody reads or marks it now
            if (tid == 0) bad_nodes[(seg & 1) ^ 1] = 0;
            if (more) {
                s = after;
                load_q(s);
            }
            // (the last scores say that all products but the last two are done,
            // so that of either barrier only the last phase can be open)
            wait(&pv[(i - 1) & 1], (i - 1) >> 1);
            at_after();
            put_tile<KIND, DP>(A, share, done, tbase + lanes + T_O, r, node, nodes_bad & mask, ref, tot, 0, DP);
            at_before();
            __syncwarp();
            if (lane == 0) at_arrive(&of);
            if (!more) break;
        }
    }

    at_before();
    __syncthreads();
    at_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tbase) : "memory");
    if (threadIdx.x == 0 && *gone && A.status) atomicOr(A.status, int(SPEC_BADBIT_TIMEOUT));
}

template <int KIND, int DP>
cudaError_t launch_tiles(const AttnLaunch& L) {
    using S = TilesShape<DP>;
    static bool ready[64] = {};  // per device; setting it twice does no harm
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev]) {
        e = cudaFuncSetAttribute(k_attn_tiles<KIND, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(S::SMEM));
        if (e != cudaSuccess) return e;
        ready[dev] = true;
    }
    e = launch_behind(k_attn_tiles<KIND, DP>, dim3(unsigned(L.ctas)), S::THREADS, S::SMEM, L.st, L.mk, L.mv, L.A);
    return e == cudaSuccess ? launch_attn_join(L, DP) : e;
}

}  // namespace sv
