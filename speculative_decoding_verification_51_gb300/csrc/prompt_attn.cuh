// prompt_attn.cuh -- k_prompt: causal attention over packed prompts on the tcgen05 tensor
// cores.
//
// For query i of a prompt with n queries over m keys, keys j <= i + m - n (and, with a
// window, j > i + m - n - window): o = sum_j 2^(c s_j - r) v_j / sum_j 2^(c s_j - r), s = q k,
// in one pass over the keys with a running reference r.
//
// A CTA takes one item: two tiles of 128 rows (one of a wide head), whose softmax and
// products take turns: while the weights of one are made, the tensor cores work for the other.
//   warp 0        TMA: the rows of Q, then K and V of 128 keys by turns through one ring
//   warp 1        one thread issues the products: S = Q K^T into TMEM, O += P V with
//                 P in TMEM, over the columns that S had
//   warps 2, 3    in tiles of keys that some row does not see whole: V's rows past the prompt, and
//                 values that are not finite, become zero (a weight of zero would not hide them)
//   warps 4..     softmax, one row a thread: the scores in registers, the weights back to
//                 TMEM as 16 bits, the row's reference and total in registers; then the row of O
//
// As in k_attn_tiles the reference is raised only when a score passes it by some octaves, so
// that O is seldom rescaled; weights are rounded to the queries' type, relative.
#pragma once

#include "prompt.cuh"

namespace sv {
namespace {

template <int DP>
struct PromptShape {
    static constexpr int MT = DP <= 128 ? 2 : 1;          // row tiles
    static constexpr int CH = DP < 128 ? DP : 128;        // channels of a stage
    static constexpr int CHUNKS = DP / CH;                // stages of a tile of keys
    static constexpr int STAGE = CH / 64 * 16384;         // bytes
    static constexpr int Q_TILE = DP / 64 * 16384;
    static constexpr int STAGES = DP == 64 ? 8 : 5;
    static constexpr size_t SMEM = 1024 + size_t(MT) * Q_TILE + size_t(STAGES) * STAGE;
    static_assert(SMEM + 1024 <= 232448, "shared memory");
    static constexpr int THREADS = 128 + MT * 128;
    static constexpr int HIDDEN = 8;  // tiles of keys not seen whole, at most: two at either end of a row tile's
};

template <bool F16, int DP>
__global__ void __launch_bounds__(PromptShape<DP>::THREADS, 1)
    k_prompt(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
             const __grid_constant__ CUtensorMap mv, const __grid_constant__ PromptArgs A) {
    using S = PromptShape<DP>;
    constexpr int MT = S::MT, ST = S::STAGES, CHUNKS = S::CHUNKS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sm_q = smem;
    uint8_t* ring = smem + MT * S::Q_TILE;
    __shared__ __align__(8) uint64_t full[ST], empty[ST];
    __shared__ __align__(8) uint64_t qf[MT], sf[2], pf[2], pv, of[MT], near[S::HIDDEN], clean[S::HIDDEN], fin;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    __shared__ uint32_t bad[S::HIDDEN][4];  // tokens with values that are not finite
    __shared__ int bad_at[S::HIDDEN];       // in which tile of keys
    __shared__ int bad_any, bad_tiles;

    begin_after_previous();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned unit = blockIdx.x;
    const int sub = MT == 1 ? int(unit & 1u) : 0;  // a wide head: which of the item's row tiles
    if (MT == 1) unit >>= 1;
    const int rank = int(unit / unsigned(A.Hkv)), h = int(unit - unsigned(rank) * unsigned(A.Hkv));
    // a plan that was made for other sizes leads nowhere
    if (rank >= A.plan->items || A.plan->T != A.T || A.plan->M != A.M || A.plan->tokens != A.tokens) return;
    PromptItem item = reinterpret_cast<const PromptItem*>(A.plan + 4)[rank];
    if (MT == 1 && sub) {
        item.q0 += A.tokens;
        item.n -= A.tokens;
        item.last += A.tokens;
        if (item.n <= 0) return;
    }
    // Tile t's tokens and the tiles of keys [lo, hi) that its rows see.
    auto tokens_of = [&](int t) { return max(0, min(A.tokens, item.n - t * A.tokens)); };
    int lo[MT], hi[MT];
    int j0 = 0x7fffffff, j1 = 0;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int n = tokens_of(t), first = item.last + t * A.tokens;
        lo[t] = A.window ? max(0, first - A.window + 1) / PROMPT_KEYS : 0;
        hi[t] = n ? (first + n + PROMPT_KEYS - 1) / PROMPT_KEYS : 0;
        if (first + n <= 0) hi[t] = 0;
        if (hi[t] > lo[t]) {
            j0 = min(j0, lo[t]);
            j1 = max(j1, hi[t]);
        } else {
            lo[t] = hi[t] = 0;
        }
    }
    if (j1 == 0) j0 = 0;
    auto in = [&](int t, int j) { return j >= lo[t] && j < hi[t]; };
    // whether some row of tile t does not see all of tile j of its keys
    auto hidden = [&](int t, int j) {
        const int first = item.last + t * A.tokens;
        return j * PROMPT_KEYS + PROMPT_KEYS - 1 > first ||
               (A.window && j * PROMPT_KEYS < first + tokens_of(t) - A.window);
    };
    auto any_hidden = [&](int j) {
        return (in(0, j) && hidden(0, j)) || (MT == 2 && in(MT - 1, j) && hidden(MT - 1, j));
    };

    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sf[i], 1);
            mbar_init(&pf[i], 4);
        }
        for (int i = 0; i < MT; ++i) {
            mbar_init(&qf[i], 1);
            mbar_init(&of[i], 1);
        }
        mbar_init(&pv, 1);
        for (int i = 0; i < S::HIDDEN; ++i) {
            mbar_init(&near[i], 1);
            mbar_init(&clean[i], 2);
        }
        mbar_init(&fin, 1);
        abort_flag = 0;
        bad_any = 0;
        fence_mbarrier_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_base))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    at_before();
    __syncthreads();
    at_after();
    const uint32_t tbase = tmem_base;
    constexpr uint32_t T_O = 256;  // S buffers at 0 and 128 (and P over them), then O
    volatile int* gone = &abort_flag;
    // a bounded wait; once one has run out nobody waits any more
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity & 1u) || *gone) return;
        if (!at_wait_bounded(bar, parity & 1u, AT_WAIT_NS)) *gone = 1;
    };

    if (warp == 0) {
        // ---- copies
        if (lane == 0) {
            uint32_t i = 0;  // stages so far
            auto query = [&](int t) {
                if (hi[t] <= lo[t]) return;
                mbar_arrive_expect_tx(&qf[t], uint32_t(DP / 64 * 128 * A.tokens * A.G));
                for (int c = 0; c < DP / 64; ++c)
                    tma_load_4d(sm_q + t * S::Q_TILE + c * 16384, &mq, c * 64, 0, h, item.q0 + t * A.tokens, &qf[t]);
            };
            auto keys = [&](const CUtensorMap* map, int j) {
                for (int c = 0; c < CHUNKS; ++c, ++i) {
                    const uint32_t st = i % ST;
                    wait(&empty[st], (i / ST) ^ 1u);
                    if (*gone) return;
                    mbar_arrive_expect_tx(&full[st], uint32_t(S::STAGE));
                    for (int x = 0; x < S::CH / 64; ++x)
                        tma_load_4d(ring + st * S::STAGE + x * 16384, map, c * S::CH + x * 64, 0, h,
                                    item.k0 + j * PROMPT_KEYS, &full[st]);
                }
            };
            query(0);
            for (int j = j0; j < j1 && !*gone; ++j) {
                keys(&mk, j);
                if (MT == 2 && j == j0) query(MT - 1);
                keys(&mv, j);
            }
            // every copy has landed before the CTA leaves (they have, unless a wait ran out)
            if (*gone) {
                for (int t = 0; t < MT; ++t)
                    if (hi[t] > lo[t]) at_wait_bounded(&qf[t], 0, AT_WAIT_NS / 8);
                for (uint32_t x = i > ST ? i - ST : 0; x < i; ++x)
                    at_wait_bounded(&full[x % ST], (x / ST) & 1u, AT_WAIT_NS / 8);
            }
        }
    } else if (warp == 1) {
        // ---- products
        if (lane == 0) {
            constexpr uint32_t id_s = at_idesc<F16>(128, false), id_o = at_idesc<F16>(S::CH, true);
            const uint32_t qa = smem_u32(sm_q), ra = smem_u32(ring);
            auto k_stage = [&](int j) { return uint32_t(j - j0) * 2 * CHUNKS; };
            auto v_stage = [&](int j) { return uint32_t(j - j0) * 2 * CHUNKS + CHUNKS; };
            auto scores = [&](int t, int j) {  // (one tile: each chunk of K is released behind its products)
                if (j == lo[t]) {
                    wait(&qf[t], 0);
                }
                const uint32_t d = tbase + (MT == 2 ? t : (j - j0) & 1) * 128;
                for (int c = 0; c < CHUNKS; ++c) {
                    const uint32_t i = k_stage(j) + c, st = i % ST;
                    wait(&full[st], i / ST);
                    at_after();
                    const uint32_t ka = ra + st * S::STAGE, q = qa + t * S::Q_TILE + c * S::STAGE;
#pragma unroll
                    for (int k = 0; k < S::CH / 16; ++k)
                        at_mma_ss(d, at_desc_k(q + (k >> 2) * 16384 + (k & 3) * 32),
                                  at_desc_k(ka + (k >> 2) * 16384 + (k & 3) * 32), id_s, c > 0 || k > 0);
                    if (MT == 1) at_commit(&empty[st]);
                }
                at_commit(&sf[MT == 2 ? t : (j - j0) & 1]);
            };
            // The cleaners are told that a tile of keys comes up (they follow no ring of their own)
            // while its softmax is under way, and waited for before its values are used.
            int cleaned = 0;
            auto tell = [&](int j) {
                const bool unclean = any_hidden(j);
                if (unclean) at_arrive(&near[cleaned]);
                return unclean;
            };
            auto sums = [&](int t, int j, bool wait_clean) {
                const uint32_t n = uint32_t(j - lo[t]);
                if (wait_clean) wait(&clean[cleaned++], 0);
                wait(&pf[MT == 2 ? t : n & 1], MT == 2 ? n : n >> 1);
                const uint32_t p = tbase + (MT == 2 ? t : (j - j0) & 1) * 128;
                for (int c = 0; c < CHUNKS; ++c) {
                    const uint32_t i = v_stage(j) + c, st = i % ST;
                    wait(&full[st], i / ST);
                    at_after();
                    const uint32_t va = ra + st * S::STAGE;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        at_mma_ts(tbase + T_O + t * DP + c * S::CH, p + k * 8, at_desc_mn(va + k * 2048), id_o,
                                  j > lo[t] || k > 0);
                    if (MT == 1) at_commit(&empty[st]);
                }
                if (MT == 1) at_commit(&pv);
                if (j + 1 == hi[t]) at_commit(&of[t]);
            };
            auto release = [&](uint32_t i) {
                for (int c = 0; c < CHUNKS; ++c) at_commit(&empty[(i + c) % ST]);
            };
            if (j1 > j0) {
                if constexpr (MT == 2) {
                    for (int t = 0; t < MT; ++t)
                        if (in(t, j0)) scores(t, j0);
                    release(k_stage(j0));
                    for (int j = j0; j < j1; ++j) {
                        bool unclean = tell(j);
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            if (in(t, j)) {
                                sums(t, j, unclean);
                                unclean = false;
                            }
                            if (in(t, j + 1)) scores(t, j + 1);
                        }
                        release(v_stage(j));
                        if (j + 1 < j1) release(k_stage(j + 1));
                    }
                } else {
                    scores(0, j0);
                    for (int j = j0; j < j1; ++j) {
                        if (j + 1 < j1) scores(0, j + 1);
                        sums(0, j, tell(j));
                    }
                }
            }
            at_commit(&fin);  // every product is done before TMEM is freed
            at_wait_bounded(&fin, 0, AT_WAIT_NS);
        }
    } else if (warp < 4) {
        // ---- values that must not meet a weight of zero
        const int tid = threadIdx.x - 64;
        int slot = 0;
        for (int j = j0; j < j1; ++j) {
            if (!any_hidden(j)) continue;
            wait(&near[slot], 0);
            if (tid < 4) bad[slot][tid] = 0;
            if (tid == 0) bad_at[slot] = j;
            asm volatile("bar.sync 2, 64;" ::: "memory");
            for (int c = 0; c < CHUNKS; ++c) {
                const uint32_t i = uint32_t(j - j0) * 2 * CHUNKS + CHUNKS + c, st = i % ST;
                wait(&full[st], i / ST);
                constexpr uint32_t EX = F16 ? 0x7c007c00u : 0x7f807f80u;
#pragma unroll 4
                for (int x = tid; x < S::STAGE / 16; x += 64) {
                    const int row = (x >> 3) & 127;
                    uint4* p = reinterpret_cast<uint4*>(ring + st * S::STAGE) + x;
                    if (j * PROMPT_KEYS + row >= item.m) {
                        *p = make_uint4(0, 0, 0, 0);
                        continue;
                    }
                    const uint4 v = *p;
                    uint32_t u[4] = {v.x, v.y, v.z, v.w};
                    bool hit = false;
#pragma unroll
                    for (int e = 0; e < 4; ++e) hit |= (u[e] & EX & 0xffffu) == (EX & 0xffffu) || (u[e] & EX) >> 16 == EX >> 16;
                    if (__builtin_expect(hit, 0)) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if ((u[e] & EX & 0xffffu) == (EX & 0xffffu)) u[e] &= 0xffff0000u;
                            if ((u[e] & EX) >> 16 == EX >> 16) u[e] &= 0xffffu;
                        }
                        *p = make_uint4(u[0], u[1], u[2], u[3]);
                        atomicOr(&bad[slot][row >> 5], 1u << (row & 31));
                        bad_any = 1;
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) at_arrive(&clean[slot]);
            ++slot;
        }
        if (tid == 0) bad_tiles = slot;
        asm volatile("bar.arrive 1, %0;" ::"r"(64 + MT * 128) : "memory");
    } else {
        // ---- softmax: row = this thread's TMEM lane
        const int t = MT == 2 ? (warp - 4) >> 2 : 0, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
        const int tok = r / A.G, g = r - tok * A.G, token = t * A.tokens + tok;
        const bool mine = tok < A.tokens && token < item.n;
        const int end = item.last + token, begin = A.window ? end - A.window + 1 : 0;  // keys it sees: [begin, end]
        const uint32_t o = tbase + lanes + T_O + t * DP;
        const float c = A.c;
        const int ja = t ? lo[MT - 1] : lo[0], jb = t ? hi[MT - 1] : hi[0];
        float ref = -INFINITY, tot = 0.f;
        for (int j = ja; j < jb; ++j) {
            const uint32_t n = uint32_t(j - ja), buf = MT == 2 ? t : n & 1;
            const uint32_t sa = tbase + lanes + buf * 128;
            wait(&sf[buf], MT == 2 ? n : n >> 1);
            at_after();
            uint32_t x[4][32];
#pragma unroll
            for (int y = 0; y < 4; ++y) at_ld32(sa + y * 32, x[y]);
#pragma unroll
            for (int y = 0; y < 4; ++y) at_ld_wait(x[y]);
            if (__builtin_expect(hidden(t, j), 0)) {
                const int above = end - j * PROMPT_KEYS, below = begin - j * PROMPT_KEYS;
#pragma unroll
                for (int y = 0; y < 4; ++y)
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const int at = y * 32 + e;
                        if (at > above || at < below) x[y][e] = 0xff800000u;
                    }
            }
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int y = 0; y < 4; ++y)
#pragma unroll
                for (int e = 0; e < 32; e += 2)
                    m4[y] = fmaxf(fmaxf(__uint_as_float(x[y][e]), __uint_as_float(x[y][e + 1])), m4[y]);
            const float top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * c;
            const bool raise = top > ref + TilesRange<F16>::SLACK;
            if (__any_sync(0xffffffffu, raise)) {
                const float to = raise ? top - TilesRange<F16>::TOP : ref;
                const float f = ref == to ? 1.f : ex2_approx(ref - to);
                ref = to;
                tot *= f;
                if (n > 0) {  // O holds sums by the old reference
                    if (MT == 1) wait(&pv, n - 1);
                    scale_rows<DP>(o, f);
                }
            }
            const float at = ref == -INFINITY ? 0.f : -ref;
            const uint64_t c2 = f2_pack(c, c), at2 = f2_pack(at, at);
            uint64_t s0 = f2_pack(0.f, 0.f), s1 = s0;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                uint32_t p[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float a, b;
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(x[y][2 * e]), __uint_as_float(x[y][2 * e + 1])), c2, at2), a, b);
                    a = ex2_approx(a);
                    b = ex2_approx(b);
                    if (e & 1) s1 = f2_add(s1, f2_pack(a, b));
                    else s0 = f2_add(s0, f2_pack(a, b));
                    p[e] = pack16<F16>(a, b);
                }
                at_st16(sa + y * 16, p);
            }
            at_st_wait();
            at_before();
            __syncwarp();
            if (lane == 0) at_arrive(&pf[buf]);
            float a, b;
            f2_unpack(f2_add(s0, s1), a, b);
            tot += a + b;
        }
        asm volatile("bar.sync 1, %0;" ::"r"(64 + MT * 128) : "memory");  // the cleaners' marks are there
        if (jb > ja) wait(&of[t], 0);
        at_after();
        const bool none = tot == 0.f || jb <= ja;
        const float inv = none ? 0.f : 1.f / tot;
        uint16_t* out = static_cast<uint16_t*>(A.out) + ((long long)(item.q0 + token) * A.Hq + h * A.G + g) * A.D;
#pragma unroll 1
        for (int d = 0; d < DP; d += 32) {
            uint32_t u[32];
            at_ld32(o + d, u);
            at_ld_wait(u);
            float f[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] = none ? 0.f : __uint_as_float(u[e]);
            if (__builtin_expect(bad_any, 0) && mine) {
                // what it sees of values that are not finite
                for (int s = 0; s < bad_tiles; ++s) {
                    if (bad_at[s] < ja || bad_at[s] >= jb) continue;
                    for (int w = 0; w < 4; ++w)
                        for (uint32_t b = bad[s][w]; b; b &= b - 1) {
                            const int key = bad_at[s] * PROMPT_KEYS + w * 32 + __ffs(b) - 1;
                            if (key > end || key < begin) continue;
                            const uint16_t* v = static_cast<const uint16_t*>(A.v) + (item.k0 + key) * A.v_token + h * A.v_head;
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (d + e < A.D) {
                                    const float z = F16 ? __half2float(reinterpret_cast<const __half*>(v)[d + e])
                                                        : __uint_as_float(uint32_t(v[d + e]) << 16);
                                    if (!(fabsf(z) < INFINITY)) f[e] += z;
                                }
                        }
                }
            }
            if (mine) {
#pragma unroll
                for (int e = 0; e < 32; e += 8)
                    if (d + e < A.D) {
                        uint32_t w[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) w[y] = pack16<F16>(f[e + 2 * y] * inv, f[e + 2 * y + 1] * inv);
                        if (none) w[0] = w[1] = w[2] = w[3] = 0;
                        *reinterpret_cast<uint4*>(out + d + e) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
            }
            __syncwarp();
        }
        if (mine && A.lse)
            A.lse[(long long)(item.q0 + token) * A.Hq + h * A.G + g] =
                none ? -INFINITY : (ref + log2f(tot)) * 0.6931471805599453f;
    }

    at_before();
    __syncthreads();
    at_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tbase) : "memory");
    if (threadIdx.x == 0 && *gone && A.status) atomicOr(A.status, int(SPEC_BADBIT_TIMEOUT));
}

template <bool F16, int DP>
cudaError_t launch_prompt_of(const PromptLaunch& L) {
    using S = PromptShape<DP>;
    static bool ready[64] = {};  // per device; setting it twice does no harm
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev]) {
        e = cudaFuncSetAttribute(k_prompt<F16, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(S::SMEM));
        if (e != cudaSuccess) return e;
        ready[dev] = true;
    }
    return launch_behind(k_prompt<F16, DP>, dim3(L.ctas), S::THREADS, S::SMEM, L.st, L.mq, L.mk, L.mv, L.A);
}

template <bool F16>
cudaError_t launch_prompt_any(const PromptLaunch& L) {
    return L.A.D <= 64 ? launch_prompt_of<F16, 64>(L) : L.A.D <= 128 ? launch_prompt_of<F16, 128>(L) : launch_prompt_of<F16, 256>(L);
}

}  // namespace
}  // namespace sv
