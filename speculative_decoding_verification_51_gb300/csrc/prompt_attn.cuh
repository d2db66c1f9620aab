// prompt_attn.cuh -- k_prompt: causal attention over packed prompts on the tcgen05 tensor
// cores.
//
// For query i of a prompt with n queries over m keys, keys j <= i + m - n (and, with a
// window, j > i + m - n - window): o = sum_j 2^(c s_j - r) v_j / sum_j 2^(c s_j - r), s = q k,
// in one pass over the keys with a running reference r.
//
// One CTA an SM, items one after another without a break between them.  An item is two tiles of 128
// rows (one of a wide head), whose softmax and products take turns: while the weights of one are
// made, the tensor cores work for the other.
//   warp 0        TMA: the rows of Q, then K and V of 128 keys by turns through one ring, and behind an
//                 item's last V a stage a row tile for its rows of O
//   warps 1, 2    one thread of a warp a row tile issues the products: S = Q K^T into TMEM, O += P V with
//                 P in TMEM, over the columns that S had.  (A wide head has warp 1 alone.)
//   warp 3        in tiles of keys that some row does not see whole: V's rows past the prompt, and
//                 values that are not finite, become zero (a weight of zero would not hide them); what a row
//                 sees of such values is added to its sums at the end
//   warps 4..     softmax, one row a thread: the scores in registers, the weights back to
//                 TMEM as 16 bits, the row's reference and total in registers; then the row of O
//
// As in k_attn_tiles the reference is raised only when a score passes it by some octaves, so
// that O is seldom rescaled; weights are rounded to the queries' type, relative.
//
// 16001 tokens of 32 query heads over 8 of 128 channels take 1380 us (1520 TFLOP/s, 0.78 of the measured burst rate,
// 0.88 of the sustained one), and 1270 in ten passes over the same inputs, which end before the power limit lowers the clock
// (1.99 GHz, then 1.82 to 1.85); 8192 of 32 over 32 heads 374.  What bounds it: of some 3020 cycles a step (a tile of
// keys for both row tiles) the tensor cores need 2048, and the scores' products, both operands in shared memory, want
// all of its 128 bytes a cycle; the rest is what the two tiles' softmax and products wait for one another.
// Heads of 256 channels run at 1180 TFLOP/s (one row tile: its softmax and products wait for one another), of 64 at
// 820 (the softmax of a tile takes as long, its products half).  At 168 registers a thread some 50 bytes spill.
#pragma once

#include <algorithm>

#include "prompt.cuh"
#include "ring.cuh"

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

// Descriptors by their low words: the high one is a constant of the 128-byte swizzle (8 rows
// 1024 bytes apart), and what follows within an operand adds to the address alone.  The thread that
// issues the products has some 2000 cycles a step for all of its instructions.
constexpr uint32_t DESC_HIGH = (1024 >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_k(uint32_t a) { return (a >> 4) | 1u << 16; }
__device__ __forceinline__ uint32_t desc_mn(uint32_t a) { return (a >> 4) | uint32_t(16384 >> 4) << 16; }
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(DESC_HIGH)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(DESC_HIGH)
        : "memory");
}

// A value that is the same in all lanes, so that the compiler knows it: what the products are
// given then stays in uniform registers (moved there for each product, an issue took 60 cycles).
template <class T>
__device__ __forceinline__ T uniform(T x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ bool elect_one() {
    uint32_t on;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(on));
    return on != 0;
}

// A place in the ring.
template <int ST>
struct RingAt {
    uint32_t st = 0, phase = 0;
    __device__ __forceinline__ void next() {
        if (++st == ST) {
            st = 0;
            phase ^= 1u;
        }
    }
    __device__ __forceinline__ void skip(uint32_t n) {
        const uint32_t x = st + n, q = x / ST;
        st = x - q * ST;
        phase ^= q & 1u;
    }
};

// A CTA's items: the list's places c, 2 n - 1 - c, 2 n + c, ... of n CTAs.  The list has the
// longest first, so that every CTA's share comes out alike.
__device__ __forceinline__ long long place_of(int round) {
    return (long long)round * gridDim.x + (round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

// One item as the roles see it: tile t's rows are tokens [t * tokens, ...), and its rows see the
// tiles of keys [lo[t], hi[t]); [j0, j1) are those of all.
template <int DP>
struct PromptWork {
    static constexpr int MT = PromptShape<DP>::MT;
    int q0, n, k0, last, m, h;
    int lo[MT], hi[MT], j0, j1;
    int up[MT], down[MT];  // tile t's rows see tiles j of keys with down[t] <= j < up[t] whole
    int all_up, all_down;  // and both of them these

    // The item's words as they lie in the plan (any place's: of one past the end, the last one's)
    struct Words {
        int4 x;
        int m, h, sub;
    };
    __device__ __forceinline__ static Words words(const PromptArgs& A, long long place, long long total) {
        Words r;
        uint32_t at = uint32_t(min(place, total - 1));
        r.sub = 0;
        if (MT == 1) {  // a wide head: which of the item's row tiles
            r.sub = int(at & 1);
            at >>= 1;
        }
        const uint32_t rank = at / uint32_t(A.Hkv);
        r.h = int(at - rank * uint32_t(A.Hkv));
        const int4* p = reinterpret_cast<const int4*>(A.plan + 4) + 2ll * rank;
        r.x = __ldg(p);
        r.m = __ldg(&p[1].x);
        return r;
    }
    __device__ __forceinline__ PromptWork() {}
    __device__ __forceinline__ PromptWork(const PromptArgs& A, const Words& r) {
        h = r.h;
        m = r.m;
        q0 = r.x.x + r.sub * A.tokens;
        n = r.x.y - r.sub * A.tokens;
        k0 = r.x.z;
        last = r.x.w + r.sub * A.tokens;
        j0 = all_up = 0x7fffffff;
        j1 = all_down = 0;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int tn = max(0, min(A.tokens, n - t * A.tokens)), first = last + t * A.tokens;
            lo[t] = A.window ? max(0, first - A.window + 1) / PROMPT_KEYS : 0;
            hi[t] = tn && first + tn > 0 ? (first + tn + PROMPT_KEYS - 1) / PROMPT_KEYS : 0;
            up[t] = max(0, first + 1) / PROMPT_KEYS;
            down[t] = A.window ? (max(0, first + tn - A.window) + PROMPT_KEYS - 1) / PROMPT_KEYS : 0;
            if (hi[t] > lo[t]) {
                j0 = min(j0, lo[t]);
                j1 = max(j1, hi[t]);
                all_up = min(all_up, up[t]);
                all_down = max(all_down, down[t]);
            } else {
                lo[t] = hi[t] = 0;
            }
        }
        if (j1 == 0) j0 = 0;
    }
    __device__ __forceinline__ bool any_hidden(int j) const { return j >= all_up || j < all_down; }
    // stages of the ring, behind the item's values, for its rows of O on their way out: of row tiles
    // that see something (the others' zeros go out directly)
    __device__ __forceinline__ uint32_t out_stages() const {
        uint32_t n = 0;
#pragma unroll
        for (int t = 0; t < MT; ++t) n += hi[t] > lo[t] ? PromptShape<DP>::CHUNKS : 0;
        return n;
    }
};

template <bool F16, int DP>
__global__ void __launch_bounds__(PromptShape<DP>::THREADS, 1)
    k_prompt(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
             const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo,
             const __grid_constant__ PromptArgs A) {
    using S = PromptShape<DP>;
    using Work = PromptWork<DP>;
    constexpr int MT = S::MT, ST = S::STAGES, C = S::CHUNKS;
    constexpr int CLEANERS = 3 - MT;  // warps
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sm_q = smem;
    uint8_t* ring = smem + MT * S::Q_TILE;
    __shared__ __align__(8) uint64_t full[ST], empty[ST];  // of the ring
    __shared__ __align__(8) uint64_t qf[MT], qe[MT];       // a tile's queries there, used
    __shared__ __align__(8) uint64_t sf[2], pf[2][2];      // a buffer's scores there, its weights of either half of the keys
    __shared__ __align__(8) uint64_t of[MT], oe[MT];       // a tile's sums there, read
    __shared__ __align__(8) uint64_t pv, near, clean, fin;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    __shared__ uint32_t copied;  // stages that warp 0 has begun to fill
    __shared__ int busy[2][4];  // a row tile's softmax at work, by the quarter of the SM that it shares with the other's
    // values that are not finite, by the parity of the CTA's item: in which tiles of keys, which tokens
    __shared__ uint32_t bad[2][S::HIDDEN][4];
    __shared__ int bad_at[2][S::HIDDEN], bad_tiles[2], bad_item[2];  // (bad_item: whose they are)

    begin_after_previous();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // a plan that was made for other sizes leads nowhere
    const bool fits = A.plan->T == A.T && A.plan->M == A.M && A.plan->tokens == A.tokens;
    const long long total = fits ? (long long)A.plan->items * A.Hkv * (MT == 1 ? 2 : 1) : 0;
    if (place_of(0) >= total) return;  // (the first round: no later one has an item either)

    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], MT);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sf[i], 1);
            mbar_init(&pf[i][0], 4);
            mbar_init(&pf[i][1], 4);
            bad_tiles[i] = 0;
            bad_item[i] = -1;
        }
        for (int i = 0; i < MT; ++i) {
            mbar_init(&qf[i], 1);
            mbar_init(&qe[i], 1);
            mbar_init(&of[i], 1);
            mbar_init(&oe[i], 4);
        }
        mbar_init(&pv, 1);
        mbar_init(&near, MT);
        mbar_init(&clean, CLEANERS);
        mbar_init(&fin, MT);
        abort_flag = 0;
        copied = 0;
        for (int i = 0; i < 8; ++i) busy[i >> 2][i & 3] = 0;
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
    // A bounded wait; once one has run out nobody waits any more.  Whoever was not waited for to the
    // end (`lost`) leaves its loop, warps that meet at a barrier together.  Until then a warp may
    // arrive at barriers that it had to wait for first, so arrivals are single ones (of several at once
    // some could be more than are pending, which is undefined), and at `full` and `qf`, which count
    // bytes too, warp 0 alone arrives, behind a wait that was not cut short.
    bool lost = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity & 1u)) return;
        if (*gone || !at_wait_bounded(bar, parity & 1u, AT_WAIT_NS)) {
            *gone = 1;
            lost = true;
        }
    };
    // For what may be many steps ahead, as many as there are keys (an item's first tile that is not seen whole; the
    // next item's scores for a row tile that has nothing to do for this one): what is bounded is the time in
    // which no stage is copied, of which a step has several.  (All waits in this form, whose code is longer:
    // 32 prompts of 20 to 2000 tokens 402 us, 8192 tokens of 256 channels 505; in this way 385 and 467.)
    volatile uint32_t* moved = &copied;
    auto wait_long = [&](uint64_t* bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity & 1u)) return;
        if (!wait_while_moving([&]() { return at_try_wait(bar, parity & 1u); }, [&]() { return *gone != 0; }, [&]() { return *moved; },
                               []() { return globaltimer_ns(); }, AT_WAIT_NS)) {
            *gone = 1;
            lost = true;
        }
    };
    // a barrier of `n` threads: whether it is lost to any of them
    auto any_lost = [&](int id, int n) {
        uint32_t any;
        asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                     : "=r"(any)
                     : "r"(uint32_t(lost)), "r"(id), "r"(n)
                     : "memory");
        return any != 0;
    };

    if (warp < 4) {
    // (the launch's 384 x 168 registers: 128 x 88 and 256 x 208)
    if constexpr (MT == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 0) {
        // ---- copies
        if (lane == 0) {
            uint32_t i = 0, uses[MT] = {};  // stages, and queries of a tile, so far
            auto ahead = Work::words(A, place_of(0), total);
            for (int round = 0; place_of(round) < total && !*gone; ++round) {
                const Work w(A, ahead);
                ahead = Work::words(A, place_of(round + 1), total);
                auto query = [&](int t) {
                    if (w.hi[t] <= w.lo[t]) return;
                    wait(&qe[t], uses[t] ^ 1u);
                    if (*gone) return;
                    mbar_arrive_expect_tx(&qf[t], uint32_t(DP / 64 * 128 * A.tokens * A.G));
                    for (int c = 0; c < DP / 64; ++c)
                        tma_load_4d(sm_q + t * S::Q_TILE + c * 16384, &mq, c * 64, 0, w.h, w.q0 + t * A.tokens, &qf[t]);
                    ++uses[t];
                };
                auto keys = [&](const CUtensorMap* map, int j) {
                    for (int c = 0; c < C; ++c) {
                        const uint32_t st = i % ST;
                        wait(&empty[st], (i / ST) ^ 1u);
                        if (*gone) return;
                        mbar_arrive_expect_tx(&full[st], uint32_t(S::STAGE));
                        for (int x = 0; x < S::CH / 64; ++x)
                            tma_load_4d(ring + st * S::STAGE + x * 16384, map, c * S::CH + x * 64, 0, w.h,
                                        w.k0 + j * PROMPT_KEYS, &full[st]);
                        ++i;
                    }
                };
                query(0);
                for (int j = w.j0; j < w.j1 && !*gone; ++j) {
                    keys(&mk, j);
                    if (MT == 2 && j == w.j0) query(MT - 1);
                    keys(&mv, j);
                }
                for (uint32_t n = w.out_stages(); n && !*gone; --n) {
                    const uint32_t st = i % ST;
                    wait(&empty[st], (i / ST) ^ 1u);
                    if (*gone) break;
                    at_arrive(&full[st]);
                    *moved = ++i;
                }
            }
            // every copy has landed before the CTA leaves, whoever used it
            for (int t = 0; t < MT; ++t)
                if (uses[t]) at_wait_bounded(&qf[t], (uses[t] - 1) & 1u, AT_WAIT_NS / 8);
            for (uint32_t x = i > ST ? i - ST : 0; x < i; ++x)
                at_wait_bounded(&full[x % ST], (x / ST) & 1u, AT_WAIT_NS / 8);
        }
    } else if (warp <= MT) {
        // ---- products, a warp a row tile: what one waits for and sends out of turn (some 600 cycles
        // a step) is hidden behind the other's.  A step is a tile of keys of an item; the scores of the next
        // one, which may be the next item's, are issued behind the sums of this one (ahead of
        // them where there is one row tile, which has two buffers).
        constexpr uint32_t id_s = at_idesc<F16>(128, false), id_o = at_idesc<F16>(S::CH, true);
        const int t = MT == 2 ? uniform(warp) - 1 : 0;
        const uint32_t qd = desc_k(smem_u32(sm_q)) + uint32_t(t * S::Q_TILE >> 4);
        const uint32_t kd = desc_k(smem_u32(ring)), vd = desc_mn(smem_u32(ring));
        const uint32_t t_s = uniform(tbase) + t * 128, t_o = t_s + T_O + t * (DP - 128);
        const bool leader = elect_one();
        RingAt<ST> ks, vs;                    // the next scores' keys, the next sums' values
        uint32_t queries = 0, outs = 0;       // uses of the tile's queries and sums so far
        uint32_t weights = 0;                 // and its tiles of weights
        uint32_t buf = 0;                     // one tile: the next scores' buffer
        bool unread = false;                  // sums that softmax may not have read yet
        uint32_t cleaned = 0;
        // (Both warps wait for every stage, used or not: a phase that is waited for is never two behind.)
        auto scores = [&](bool in, bool first, bool last) {
            if (in && first) wait(&qf[t], queries++);
            const uint32_t d = t_s + buf * 128;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                wait(&full[ks.st], ks.phase);
                if (in && leader) {
                    at_after();
                    const uint32_t k0 = kd + ks.st * (S::STAGE >> 4), q = qd + (c * S::STAGE >> 4);
#pragma unroll
                    for (int k = 0; k < S::CH / 16; ++k)
                        mma_ss(d, q + (k >> 2) * 1024 + (k & 3) * 2, k0 + (k >> 2) * 1024 + (k & 3) * 2, id_s, c > 0 || k > 0);
                    if (c == C - 1) at_commit(&sf[MT == 2 ? t : buf]);
                    at_commit(&empty[ks.st]);
                } else if (leader) {
                    at_arrive(&empty[ks.st]);
                }
                ks.next();
            }
#pragma unroll
            for (int c = 0; c < C; ++c) ks.next();
            if (in && last && leader) at_commit(&qe[t]);
            if (MT == 1) buf ^= 1u;
        };
#pragma unroll
        for (int c = 0; c < C; ++c) vs.next();
        // `unclean`: the cleaners, who were told when the weights were under way, have to be done
        auto sums = [&](bool in, bool first, bool last, bool unclean) {
            if (unclean && leader) at_arrive(&near);
            const uint32_t p = t_s + (MT == 2 ? 0u : (weights & 1u) * 128);
            if (in) {
                if (first && unread) wait(&oe[t], outs - 1);  // what the last item left has been read
            }
            if (unclean) wait(&clean, cleaned++);
            auto weighed = [&](int half) { wait(&pf[MT == 2 ? t : weights & 1u][half], MT == 2 ? weights : weights >> 1); };
#pragma unroll
            for (int c = 0; c < C; ++c) {
                wait(&full[vs.st], vs.phase);
                const uint32_t v0 = vd + vs.st * (S::STAGE >> 4);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (in && c == 0) weighed(half);
                    if (in && leader) {
                        at_after();
#pragma unroll
                        for (int k = 4 * half; k < 4 * half + 4; ++k)
                            mma_ts(t_o + c * S::CH, p + k * 8, v0 + k * 128, id_o, !first || k > 0);
                    }
                }
                if (in && leader) {
                    if (c == C - 1 && last) at_commit(&of[t]);
                    at_commit(&empty[vs.st]);
                } else if (leader) {
                    at_arrive(&empty[vs.st]);
                }
                vs.next();
            }
#pragma unroll
            for (int c = 0; c < C; ++c) vs.next();
            if (MT == 1 && leader) at_commit(&pv);
            if (in) ++weights;
            if (in && last) {
                ++outs;
                unread = true;
            }
        };
        int round = 0;
        // the next item with a step, from `round` on: its steps, the tile's, and which are not seen whole
        struct Steps {
            int j0, j1, lo, hi, up, down;
            uint32_t outs;
        };
        auto next_of = [&](Steps& x) {
            while (place_of(round) < total) {
                const Work w(A, Work::words(A, place_of(round++), total));
                x = {uniform(w.j0), uniform(w.j1), uniform(t ? w.lo[MT - 1] : w.lo[0]), uniform(t ? w.hi[MT - 1] : w.hi[0]),
                     uniform(w.all_up), uniform(w.all_down), uniform(w.out_stages())};
                if (x.j1 > x.j0) return true;
            }
            return false;
        };
        auto scores_of = [&](const Steps& x, int j) { scores(j >= x.lo && j < x.hi, j == x.lo, j + 1 == x.hi); };
        auto sums_of = [&](const Steps& x, int j) {
            sums(j >= x.lo && j < x.hi, j == x.lo, j + 1 == x.hi, j >= x.up || j < x.down);
        };
        Steps w, after;
        bool more = next_of(w);
        if (more) scores_of(w, w.j0);
        while (more && !__any_sync(0xffffffffu, lost)) {
            const bool next = next_of(after);
            int j = w.j0;
            for (; j + 1 < w.j1; ++j) {
                if (__any_sync(0xffffffffu, lost)) break;
                if (MT == 1) scores_of(w, j + 1);
                sums_of(w, j);
                if (MT == 2) scores_of(w, j + 1);
            }
            // (an item's end is alike for one row tile: its values, rows of O and the next keys, all at
            // once, are more than the ring holds)
            sums_of(w, j);
            ks.skip(w.outs);
            vs.skip(w.outs);
            if (next) scores_of(after, after.j0);
            // (the marks of an item are kept for one more: so whoever reads the last but one's is done)
            if (unread && !w.hi) {
                wait(&oe[t], outs - 1);
                unread = false;
            }
            w = after;
            more = next;
        }
        if (leader) at_commit(&fin);  // every product is done before TMEM is freed
        at_wait_bounded(&fin, 0, AT_WAIT_NS);
    } else {
        // ---- values that must not meet a weight of zero
        constexpr int N = CLEANERS * 32;
        const int tid = int(threadIdx.x) - (128 - N);
        uint32_t told = 0;
        RingAt<ST> vs;
#pragma unroll
        for (int c = 0; c < C; ++c) vs.next();
        int gen = 0;
        bool left = false;
        auto ahead = Work::words(A, place_of(0), total);
        for (int round = 0; place_of(round) < total && !left; ++round) {
            const Work w(A, ahead);
            ahead = Work::words(A, place_of(round + 1), total);
            int slot = 0;
            if (w.j1 <= w.j0) continue;
            for (int j = w.j0; j < w.j1; ++j) {
                const RingAt<ST> first = vs;
#pragma unroll
                for (int c = 0; c < 2 * C; ++c) vs.next();
                if (!w.any_hidden(j)) continue;
                wait_long(&near, told++);
                if (slot == 0 && tid == 0) bad_tiles[gen] = 0;
                if (tid < 4) bad[gen][slot][tid] = 0;
                left = any_lost(2, N);
                if (left) break;
                RingAt<ST> at = first;
                const int rows = w.m - j * PROMPT_KEYS;  // of the prompt
                // (keys that every row sees may hold anything: the first ones, but for a window's end)
                const int from = j < w.all_down ? 0 : min(max(w.last + 1 - j * PROMPT_KEYS, 0), PROMPT_KEYS);
                for (int c = 0; c < C; ++c, at.next()) {
                    wait(&full[at.st], at.phase);
#pragma unroll 1
                    for (int half = 0; half < S::CH / 64; ++half) {
                        uint4* part = reinterpret_cast<uint4*>(ring + at.st * S::STAGE + half * 16384);  // 8 of a row
                        for (int x = max(rows, from) * 8 + tid; x < PROMPT_KEYS * 8; x += N) part[x] = make_uint4(0, 0, 0, 0);
                        // an exponent of all ones carries into the bit above it
                        constexpr uint32_t EX = F16 ? 0x7c007c00u : 0x7f807f80u, ONE = F16 ? 0x04000400u : 0x00800080u;
                        const int end = min(rows, PROMPT_KEYS) * 8;
#pragma unroll 1
                        for (int x0 = from * 8 + tid; x0 < end; x0 += 8 * N) {
                            uint32_t hit = 0;
                            uint4 v[8];
#pragma unroll
                            for (int y = 0; y < 8; ++y) v[y] = part[min(x0 + y * N, end - 1)];
#pragma unroll
                            for (int y = 0; y < 8; ++y)
                                hit |= ((v[y].x & EX) + ONE) | ((v[y].y & EX) + ONE) | ((v[y].z & EX) + ONE) | ((v[y].w & EX) + ONE);
                            if (__builtin_expect(hit & 0x80008000u, 0)) {
#pragma unroll 1
                                for (int x = x0; x < min(end, x0 + 8 * N); x += N) {
                                    uint32_t u[4] = {part[x].x, part[x].y, part[x].z, part[x].w};
                                    uint32_t some = 0;
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        const uint32_t h = ((u[e] & EX) + ONE) & 0x80008000u;
                                        some |= h;
                                        u[e] &= ~((h >> 15) * 0xffffu);
                                    }
                                    if (some) {
                                        part[x] = make_uint4(u[0], u[1], u[2], u[3]);
                                        const int row = x >> 3;
                                        atomicOr(&bad[gen][slot][row >> 5], 1u << (row & 31));
                                        bad_item[gen] = round;
                                    }
                                }
                            }
                        }
                    }
                }
                if (tid == 0) {
                    bad_at[gen][slot] = j;
                    bad_tiles[gen] = slot + 1;
                }
                ++slot;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) at_arrive(&clean);
            }
            vs.skip(w.out_stages());
            gen ^= 1;
        }
    }
    } else {
        // ---- softmax: row = this thread's TMEM lane
        if constexpr (MT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int t = MT == 2 ? (warp - 4) >> 2 : 0, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
        const int tok = r / A.G, g = r - tok * A.G, token = t * A.tokens + tok;
        const uint32_t o = tbase + lanes + T_O + t * DP;
        const float c = A.c;
        const uint64_t c2 = f2_pack(c, c);
        // The two warps that share a quarter of the SM make their weights one after the other, so that
        // the products of one row tile go on under the softmax of the other: at the same time both
        // would take as long, and both tiles' products wait for the end (1368 us against 1706).  It orders
        // nothing but time: both may begin at once, and who has waited long goes on.
        volatile int* mine_busy = &busy[t][warp & 3];
        volatile int* other_busy = &busy[MT - 1 - t][warp & 3];
        auto enter = [&]() {
            if constexpr (MT == 2) {
                for (int i = 0; i < 100 && *other_busy; ++i) {}
                *mine_busy = 1;
            }
        };
        auto leave = [&]() {
            if (MT == 2) *mine_busy = 0;
        };
        // The stage that the last rows of O were copied out of goes back to the ring behind the next
        // item's first weights, when the copy has long read it.
        RingAt<ST> lent;
        bool owed = false;
        auto release = [&]() {
            if (!owed) return;  // (one thread of the row tile's owes)
            owed = false;
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            RingAt<ST> at = lent;
            for (int x = 0; x < C; ++x, at.next())
                for (int y = 0; y < MT; ++y) at_arrive(&empty[at.st]);
        };
        RingAt<ST> os;  // the item's first stage
        uint32_t tiles = 0, outs = 0;  // tiles of weights, and finished rows, so far
        int gen = 1;
        auto ahead = Work::words(A, place_of(0), total);
        for (int round = 0; place_of(round) < total; ++round) {
            const Work w(A, ahead);
            ahead = Work::words(A, place_of(round + 1), total);
            if (w.j1 > w.j0) gen ^= 1;
            const bool mine = tok < A.tokens && token < w.n;
            const int end = w.last + token, begin = A.window ? end - A.window + 1 : 0;  // keys it sees: [begin, end]
            const int ja = t ? w.lo[MT - 1] : w.lo[0], jb = t ? w.hi[MT - 1] : w.hi[0];
            const int up = t ? w.up[MT - 1] : w.up[0], down = t ? w.down[MT - 1] : w.down[0];
            float ref = -INFINITY, tot = 0.f;
            if (jb <= ja) release();
            else wait_long(&sf[MT == 2 ? t : tiles & 1u], MT == 2 ? tiles : tiles >> 1);
            for (int j = ja; j < jb; ++j, ++tiles) {
                const uint32_t buf = MT == 2 ? t : tiles & 1u;
                const uint32_t sa = tbase + lanes + buf * 128;
                wait(&sf[buf], MT == 2 ? tiles : tiles >> 1);
                at_after();
                // (in an item of few tiles of keys the first ones and those not seen whole are not ordered: products
                // are not what they wait for.  64 prompts of 300 tokens 150 -> 125 us; in longer ones it pays
                // there too, 16001 tokens 1286 -> 1263)
                const bool masked = j >= up || j < down;
                if (jb - ja >= 8 || !(masked || j == ja)) enter();
                uint32_t x[4][32];
                float m0 = -INFINITY, m1 = -INFINITY, s0, s1;
                auto largest = [&](int y) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        m0 = fmaxf(fmaxf(__uint_as_float(x[y][e]), __uint_as_float(x[y][e + 1])), m0);
                        m1 = fmaxf(fmaxf(__uint_as_float(x[y][e + 2]), __uint_as_float(x[y][e + 3])), m1);
                    }
                };
                auto hide = [&](int y) {  // a bit for each key that the row sees
                    const int above = end - j * PROMPT_KEYS - y * 32, below = begin - j * PROMPT_KEYS - y * 32;
                    const uint32_t seen = (above >= 31 ? ~0u : above < 0 ? 0u : (2u << above) - 1u) &
                                          (below <= 0 ? ~0u : below > 31 ? 0u : ~0u << below);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!(seen & 1u << e)) x[y][e] = 0xff800000u;
                };
                // (a warp's few tokens see most pieces whole)
                auto partly = [&](int y) {
                    return !__all_sync(0xffffffffu, end - j * PROMPT_KEYS - y * 32 >= 31 && begin - j * PROMPT_KEYS - y * 32 <= 0);
                };
                uint64_t sum0, sum1, at2;
                auto weigh = [&](int y) {
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float a, b;
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(x[y][2 * e]), __uint_as_float(x[y][2 * e + 1])), c2, at2), a, b);
                        a = ex2_approx(a);
                        b = ex2_approx(b);
                        if (e & 1) sum1 = f2_add(sum1, f2_pack(a, b));
                        else sum0 = f2_add(sum0, f2_pack(a, b));
                        p[e] = pack16<F16>(a, b);
                    }
                    at_st16(sa + y * 16, p);
                };
                auto begin_sums = [&]() {
                    const float at = ref == -INFINITY ? 0.f : -ref;
                    at2 = f2_pack(at, at);
                    sum0 = sum1 = f2_pack(0.f, 0.f);
                };
                at_ld32(sa, x[0]);
                at_ld32(sa + 32, x[1]);
                at_ld_wait(x[0]);
                at_ld_wait(x[1]);
                at_ld32(sa + 64, x[2]);
                at_ld32(sa + 96, x[3]);
                // The first half's weights by the reference as it is, while the largest are sought; where
                // some row's passes it by too much (seldom, but for an item's first tile) it is
                // raised, and they are made again, from the scores in registers.
                bool again = masked || j == ja;
                if (!again) {
                    begin_sums();
                    weigh(0);
                    largest(0);
                    weigh(1);
                    largest(1);
                    at_ld_wait(x[2]);
                    at_ld_wait(x[3]);
                    largest(2);
                    largest(3);
                    again = __any_sync(0xffffffffu, lost || fmaxf(m0, m1) * c > ref + TilesRange<F16>::SLACK);
                } else {
                    if (masked) {
                        if (partly(0)) hide(0);
                        if (partly(1)) hide(1);
                    }
                    largest(0);
                    largest(1);
                    at_ld_wait(x[2]);
                    at_ld_wait(x[3]);
                    if (masked) {
                        if (partly(2)) hide(2);
                        if (partly(3)) hide(3);
                    }
                    largest(2);
                    largest(3);
                }
                if (__builtin_expect(again, 0)) {
                    if (__any_sync(0xffffffffu, lost)) {
                        at_st_wait();
                        break;
                    }
                    const float top = fmaxf(m0, m1) * c;
                    const bool raise = top > ref + TilesRange<F16>::SLACK;
                    if (__any_sync(0xffffffffu, raise)) {
                        const float to = raise ? top - TilesRange<F16>::TOP : ref;
                        const float f = ref == to ? 1.f : ex2_approx(ref - to);
                        ref = to;
                        tot *= f;
                        if (j > ja) {  // O holds sums by the old reference
                            if (MT == 1) wait(&pv, tiles - 1);
                            scale_rows<DP>(o, f);
                        }
                    }
                    begin_sums();
                    weigh(0);
                    weigh(1);
                }
                // the products with the first half of the keys begin while the second is weighed
                auto give = [&](int half) {
                    at_st_wait();
                    at_before();
                    __syncwarp();
                    if (lane == 0) at_arrive(&pf[buf][half]);
                };
                give(0);
                weigh(2);
                weigh(3);
                give(1);
                release();
                leave();
                f2_unpack(f2_add(sum0, sum1), s0, s1);
                tot += s0 + s1;
            }
            const bool none = tot == 0.f;
            const float inv = none ? 0.f : 1.f / tot;
            const uint64_t inv2 = f2_pack(inv, inv);
            uint16_t* out = static_cast<uint16_t*>(A.out) + ((long long)(w.q0 + t * A.tokens) * A.Hq + w.h * A.G) * A.D;
            // (its stages: behind the first row tile's, if that has some)
            const RingAt<ST> start = os;
            os.skip(2 * C * uint32_t(w.j1 - w.j0));
            if (t && w.hi[0] > w.lo[0]) os.skip(C);
            if (jb > ja) {
                // the row, 16 bits, to this row tile's stage, laid out as a copy by tensor map wants it
                const RingAt<ST> o0 = os;
                wait(&of[t], outs++);
                at_after();
                const bool odd = *static_cast<volatile int*>(&bad_item[gen]) == round;
                auto put = [&](const uint32_t (&u)[32], int d) {
                    float f[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(u[e]);  // (0 of a row that sees nothing)
                    if (__builtin_expect(odd, 0) && mine) {
                        // what it sees of values that are not finite
                        for (int s = 0; s < bad_tiles[gen]; ++s) {
                            const int at = bad_at[gen][s];
                            if (at < ja || at >= jb) continue;
                            for (int y = 0; y < 4; ++y)
                                for (uint32_t b = bad[gen][s][y]; b; b &= b - 1) {
                                    const int key = at * PROMPT_KEYS + y * 32 + __ffs(b) - 1;
                                    if (key > end || key < begin) continue;
                                    const uint16_t* v = static_cast<const uint16_t*>(A.v) + (w.k0 + key) * A.v_token + w.h * A.v_head;
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
                    uint8_t* row = ring + (C > 1 && d >= S::CH ? (o0.st + 1) % ST : o0.st) * S::STAGE + (d % S::CH) / 64 * 16384 + r * 128;
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        uint32_t v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float a, b;
                            f2_unpack(f2_mul(f2_pack(f[8 * y + 2 * e], f[8 * y + 2 * e + 1]), inv2), a, b);
                            v[e] = pack16<F16>(a, b);
                        }
                        *reinterpret_cast<uint4*>(row + (((d % 64 / 8 + y) ^ (r & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                };
                uint32_t u0[32], u1[32];
                at_ld32(o, u0);
                for (int x = 0; x < C; ++x, os.next()) wait(&full[os.st], os.phase);
#pragma unroll 1
                for (int d = 0; d < DP; d += 64) {
                    at_ld_wait(u0);
                    at_ld32(o + d + 32, u1);
                    put(u0, d);
                    at_ld_wait(u1);
                    if (d + 64 < DP) at_ld32(o + d + 64, u0);
                    put(u1, d + 32);
                }
                at_before();
                __syncwarp();
                if (lane == 0) at_arrive(&oe[t]);
                // a whole tile by one copy, part of one row by row
                const int rows = max(0, min(A.tokens, w.n - t * A.tokens)) * A.G;
                const bool whole = rows == A.tokens * A.G;
                if (whole) fence_proxy_async_smem();
                if (any_lost(4 + t, 128)) break;
                if (!whole) {
                    const uint32_t each = uint32_t(A.D) / 8;
                    for (uint32_t x = threadIdx.x & 127; x < uint32_t(rows) * each; x += 128) {
                        const uint32_t rr = x / each, d = (x - rr * each) * 8, tk = rr / uint32_t(A.G);
                        const uint8_t* row = ring + (C > 1 && d >= S::CH ? (o0.st + 1) % ST : o0.st) * S::STAGE + (d % S::CH) / 64 * 16384 + rr * 128;
                        *reinterpret_cast<uint4*>(out + ((long long)tk * A.Hq + (rr - tk * A.G)) * A.D + d) =
                            *reinterpret_cast<const uint4*>(row + (((d % 64 / 8) ^ (rr & 7)) << 4));
                    }
                    // (what is copied in here next comes by another path)
                    fence_proxy_async_smem();
                    asm volatile("bar.sync %0, 128;" ::"r"(4 + t) : "memory");
                }
                if ((threadIdx.x & 127) == 0) {
                    if (whole) {
                        for (int x = 0; x < DP / 64; ++x) {
                            const uint32_t st = C > 1 && x >= 2 ? (o0.st + 1) % ST : o0.st;
                            tma_store_4d(&mo, ring + st * S::STAGE + (x * 64 % S::CH) / 64 * 16384, x * 64, 0, w.h, w.q0 + t * A.tokens);
                        }
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    }
                    lent = o0;
                    owed = true;
                    if (!whole) release();
                }
            } else if (mine) {  // rows that see nothing
                for (int d = 0; d < A.D; d += 8)
                    *reinterpret_cast<uint4*>(out + ((long long)tok * A.Hq + g) * A.D + d) = make_uint4(0, 0, 0, 0);
            }
            os = start;
            os.skip(2 * C * uint32_t(w.j1 - w.j0) + w.out_stages());
            if (mine && A.lse)
                A.lse[(long long)(w.q0 + token) * A.Hq + w.h * A.G + g] =
                    none ? -INFINITY : (ref + log2f(tot)) * 0.6931471805599453f;
        }
        release();
        if ((threadIdx.x & 127) == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
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
    return launch_behind(k_prompt<F16, DP>, dim3(unsigned(std::min<long long>(L.items * (S::MT == 1 ? 2 : 1), L.sms))), S::THREADS, S::SMEM, L.st, L.mq, L.mk, L.mv, L.mo, L.A);
}

template <bool F16>
cudaError_t launch_prompt_any(const PromptLaunch& L) {
    return L.A.D <= 64 ? launch_prompt_of<F16, 64>(L) : L.A.D <= 128 ? launch_prompt_of<F16, 128>(L) : launch_prompt_of<F16, 256>(L);
}

}  // namespace
}  // namespace sv
