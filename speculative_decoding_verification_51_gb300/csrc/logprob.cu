// logprob.cu -- spec_token_logprobs: log probabilities of given tokens, the entropy of
// their distributions and the most probable alternatives, each row of logits read once.
//
// With M the largest logit, a(x) = (l(x) - M) log2(e) / T, Z = sum 2^a, and A = sum 2^a a:
//   log p(x) = (l(x) - M) / T - ln 2 log2 Z,   H = ln 2 (log2 Z - A / Z).
// Each lane keeps (M, Z, A) of what it has seen, by a maximum of its own; a larger one turns
// (Z, A) into f Z, f (A + d Z), f = 2^d, d the difference, and so do the joins of lanes,
// warps and CTAs.
//
// Alternatives.  A row is cut into groups of 512 neighbours (256 of f32), and the pass
// leaves each group's largest logit behind.  The k best tokens lie in the k groups whose largest are
// best (by value, then by place: each of those k is itself a token, and no other group's is
// as good), so that the k groups alone are read a second time for tokens as good as the k-th
// group's largest.
//
// k_logprob streams tiles of 4 KB: all tiles of all rows that are read, in order, are cut into as
// many equal shares as there are warps, so that a single row goes to many SMs and ragged ones
// load every SM alike.  A warp has two tiles on their way into shared memory (192 KB an SM; with 32 KB
// in registers, HBM ran at half its rate: 1024 rows of 151936 logits, 640 of them read, took 83 us; now 60,
// 41 of them in this kernel, whose 634 instructions a tile take 70% of the issue slots).
// It leaves a tile's (M, Z, A) and its four groups' largest in the workspace; k_logprob_join, behind
// it, joins a row's and finds its best.  Bound by HBM for many rows; by latency for few.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "cache.cuh"

namespace sv {
namespace {

constexpr int LP_THREADS = 256, LP_WARPS = LP_THREADS / 32;
constexpr int LP_CTAS = 3;  // an SM
constexpr int LP_JOIN = 128, LP_JOIN_WARPS = LP_JOIN / 32;  // threads that join a row (twelve such CTAs an SM: one round for most calls)
constexpr int LP_VECS = 256, LP_STAGES = 2;  // of a tile; of a warp's ring
constexpr int LP_BYTES = LP_VECS * 16;
constexpr size_t LP_SMEM = size_t(LP_WARPS) * LP_STAGES * LP_BYTES;
constexpr int LP_CANDIDATES = 1024, LP_SOME = 128;  // tokens that there is room for, and that are compared with one another
constexpr float LP_LOWEST = -3.4028234663852886e38f, LP_FAR = -200.f;  // 2^LP_FAR is 0 in float32

struct LogprobArgs {
    const void* logits;
    long long R, stride;
    const int32_t* rows;
    const int32_t* tokens;
    const float* temp;
    float* lp;
    float* entropy;
    int32_t* ids;
    float* top_lp;
    int32_t* list;  // entries whose rows are read, in order
    float4* part;   // [E][tiles + 1] {M, Z, A} of the tiles and, last, of the row's ends
    float4* most;   // [E][tiles + 1] largest logits of a tile's four groups; {head, tail} of the ends
    int32_t* status;
    int V, top, tiles;  // tiles of a row, at most
    long long E;
};

template <int DT>
struct Elem {
    static constexpr int SIZE = DT == SPEC_F32 ? 4 : 2, EPV = 16 / SIZE;
    using T = typename std::conditional<DT == SPEC_F32, float, typename std::conditional<DT == SPEC_F16, __half, __nv_bfloat16>::type>::type;
    static constexpr uint32_t NONE = DT == SPEC_F32 ? 0xff800000u : DT == SPEC_F16 ? 0xfc00fc00u : 0xff80ff80u;
};
template <int DT>
__device__ __forceinline__ float2 two(uint32_t w) {
    if constexpr (DT == SPEC_F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    else return make_float2(bf16_lo(w), bf16_hi(w));
}
// the EPV elements of a vector
template <int DT>
__device__ __forceinline__ void unpack(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == SPEC_F32) {
            f[i] = __uint_as_float(w[i]);
        } else {
            const float2 x = two<DT>(w[i]);
            f[2 * i] = x.x;
            f[2 * i + 1] = x.y;
        }
    }
}
// the largest of two vectors (NaN loses)
template <int DT>
__device__ __forceinline__ float largest(const uint4& a, const uint4& b) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if constexpr (DT == SPEC_F32) {
        float m = __uint_as_float(w[0]);
#pragma unroll
        for (int i = 1; i < 8; ++i) m = fmaxf(m, __uint_as_float(w[i]));
        return m;
    } else {
        auto mx = [](uint32_t x, uint32_t y) {
            uint32_t r;
            if constexpr (DT == SPEC_F16) asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
            else r = bmax2(x, y);
            return r;
        };
        const uint32_t m = mx(mx(mx(w[0], w[1]), mx(w[2], w[3])), mx(mx(w[4], w[5]), mx(w[6], w[7])));
        const float2 x = two<DT>(m);
        return fmaxf(x.x, x.y);
    }
}

// A row: its ends that no whole vector holds, and what lies between.
template <int DT>
struct Row {
    using T = typename Elem<DT>::T;
    const T* p;
    int head, vecs, tiles, tail;
    __device__ __forceinline__ Row(const LogprobArgs& A, long long row) {
        p = static_cast<const T*>(A.logits) + row * A.stride;
        head = min(A.V, int((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / Elem<DT>::SIZE);
        vecs = (A.V - head) / Elem<DT>::EPV;
        tail = A.V - head - vecs * Elem<DT>::EPV;
        tiles = (vecs + LP_VECS - 1) / LP_VECS;
    }
    __device__ __forceinline__ uint4 vec(int i) const {
        return i < vecs ? __ldg(reinterpret_cast<const uint4*>(p + head) + i)
                        : make_uint4(Elem<DT>::NONE, Elem<DT>::NONE, Elem<DT>::NONE, Elem<DT>::NONE);
    }
    // a lane's element of the ends: head by lanes 0 to 15, tail by the others; -1: none
    __device__ __forceinline__ int end_of(int lane) const {
        if (lane < 16) return lane < head ? lane : -1;
        return lane - 16 < tail ? head + vecs * Elem<DT>::EPV + lane - 16 : -1;
    }
};

struct Sums {
    float m, z, a;  // reference, sums by it
    __device__ __forceinline__ void to(float ref, float kappa) {
        const float d = fmaxf((m - ref) * kappa, LP_FAR), f = ex2_approx(d);
        a = f * fmaf(d, z, a);
        z *= f;
        m = ref;
    }
};

template <int DT, bool ENT>
struct Lane {
    Sums s{LP_LOWEST, 0.f, 0.f};
    // two vectors, whose largest the reference is not below
    __device__ __forceinline__ void take(const uint4& u, const uint4& v, float kappa) {
        float f[2 * Elem<DT>::EPV];
        unpack<DT>(u, f);
        unpack<DT>(v, f + Elem<DT>::EPV);
        const uint64_t neg = f2_pack(-s.m, -s.m), k2 = f2_pack(kappa, kappa);
        uint64_t z0 = f2_pack(0.f, 0.f), a0 = z0;
#pragma unroll
        for (int i = 0; i < Elem<DT>::EPV; ++i) {
            float x, y;
            f2_unpack(f2_mul(f2_add(f2_pack(f[2 * i], f[2 * i + 1]), neg), k2), x, y);
            const uint64_t w = f2_pack(ex2_approx(x), ex2_approx(y));
            z0 = f2_add(z0, w);
            if (ENT) a0 = f2_fma(w, f2_pack(fmaxf(x, LP_FAR), fmaxf(y, LP_FAR)), a0);  // (0 of -inf)
        }
        float x, y;
        f2_unpack(z0, x, y);
        s.z += x + y;
        if (ENT) {
            f2_unpack(a0, x, y);
            s.a += x + y;
        }
    }
    __device__ __forceinline__ void one(float l, float kappa) {
        s.to(fmaxf(s.m, l), kappa);
        const float x = (l - s.m) * kappa, w = ex2_approx(x);
        s.z += w;
        if (ENT) s.a = fmaf(w, fmaxf(x, LP_FAR), s.a);
    }
};

// The sums of a warp's lanes, in every lane.
template <bool ENT>
__device__ __forceinline__ Sums warp_join(Sums s, float kappa) {
    s.to(redux_max_f32(s.m), kappa);
    s.z = warp_sum_f(s.z);
    if (ENT) s.a = warp_sum_f(s.a);
    return s;
}

// (by the temperature itself: the difference from a logit that a mask made the lowest float
// would not be one any more in units of log2(e) / T)
__device__ __forceinline__ float log_p(float l, const Sums& s, float log_z, float T) {
    return (l - s.m) / T - 0.6931471805599453f * log_z;
}

struct Best {  // what a CTA needs for the alternatives
    float value[LP_CANDIDATES];
    int id[LP_CANDIDATES];
    int group[SPEC_MAX_TOP];
    int chosen, found;
    int digits[256], digit, left;
    bool exact;
    float round_value[LP_JOIN_WARPS];
    int round_id[LP_JOIN_WARPS];
};

// largest first, of equal ones the lowest index
__device__ __forceinline__ bool before(float v, int i, float w, int j) { return v > w || (v == w && i < j); }
__device__ __forceinline__ uint32_t ordered(float f) {  // (0 and -0 alike)
    const uint32_t u = __float_as_uint(f + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// f(value, index) for the elements of chosen groups that are at least `least`, by the warps of the
// CTA in turn.  Group 0 is the row's head, the last its tail.
template <int DT, class F>
__device__ __forceinline__ void of_groups(const LogprobArgs& A, const Row<DT>& row, const Best& B, float least, F&& f) {
    constexpr int EPV = Elem<DT>::EPV;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int U = 4;  // groups of a warp that are on their way at once
    uint4 v[U][2];
    for (int c0 = warp; c0 < B.chosen; c0 += U * LP_JOIN_WARPS) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * LP_JOIN_WARPS, g = c < B.chosen ? B.group[c] - 1 : -1;
            const bool body = g >= 0 && g < row.tiles * 4;
#pragma unroll
            for (int y = 0; y < 2; ++y) v[u][y] = row.vec(body ? g * 64 + y * 32 + lane : row.vecs);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * LP_JOIN_WARPS;
            if (c >= B.chosen) break;
            const int g = B.group[c] - 1;
            if (g < 0 || g >= row.tiles * 4) {
                const int e = row.end_of(lane);
                if (e >= 0 && (lane < 16) == (g < 0) && to_f32(row.p[e]) >= least) f(to_f32(row.p[e]), e);
                continue;
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int i = g * 64 + y * 32 + lane;
                if (i >= row.vecs || !(largest<DT>(v[u][y], v[u][y]) >= least)) continue;
                float x[EPV];
                unpack<DT>(v[u][y], x);
#pragma unroll
                for (int e = 0; e < EPV; ++e)
                    if (x[e] >= least) f(x[e], row.head + i * EPV + e);
            }
        }
    }
}

// The largest bound that `top` of the keys reach which each(f) gives f, eight bits after eight, until as
// many as wanted reach it (then `exact`: those at or above it; else those above it and `want` of those at
// it).  False where there are fewer: then all of them.  (All of the CTA.)
template <int LAST, class F>
__device__ __forceinline__ bool reach(Best& B, int top, F&& each, uint32_t& bound, int& want, bool& exact) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    bound = 0;  // the digits so far
    want = top;
    exact = false;
    for (int shift = 24; shift >= LAST && !exact; shift -= 8) {
        for (int i = threadIdx.x; i < 256; i += LP_JOIN) B.digits[i] = 0;
        __syncthreads();
        each([&](uint32_t k) {
            if (shift == 24 || (k ^ bound) >> (shift + 8) == 0) atomicAdd(&B.digits[k >> shift & 255u], 1);
        });
        __syncthreads();
        if (warp == 0) {  // from the largest digit down, eight a lane
            int n[8], all = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                n[i] = B.digits[255 - lane * 8 - i];
                all += n[i];
            }
            int sum = all;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += y;
            }
            const unsigned there = __ballot_sync(0xffffffffu, sum >= want);
            if (there == 0) {
                if (lane == 0) B.digit = -1;
            } else if (lane == __ffs(there) - 1) {
                int before = sum - all, d = 255 - lane * 8, i = 0;
                while (before + n[0] < want && i < 7) {
                    before += n[0];
#pragma unroll
                    for (int x = 0; x < 7; ++x) n[x] = n[x + 1];
                    --d;
                    ++i;
                }
                B.digit = d;
                B.left = want - before;
                B.exact = before + n[0] == want;
            }
        }
        __syncthreads();
        if (B.digit < 0) return false;
        bound |= uint32_t(B.digit) << shift;
        want = B.left;
        exact = B.exact;
        __syncthreads();
    }
    return true;
}

// the least float whose key is `bound` or more (none of -inf)
__device__ __forceinline__ float float_of(uint32_t bound) {
    const uint32_t u = max(bound, ordered(LP_LOWEST));
    return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

// The alternatives of a row (all of the CTA); most(g): the largest logit of its group g.
template <int DT, class F>
__device__ __forceinline__ void best_tokens(const LogprobArgs& A, const Row<DT>& row, Best& B, F&& most, const Sums& s, float T,
                                            long long e) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = row.tiles * 4 + 2;
    const float log_z = log2f(s.z);
    // (bf16 has no more bits than two digits hold, f16 as float no more than three)
    constexpr int LAST = DT == SPEC_BF16 ? 16 : DT == SPEC_F16 ? 8 : 0;
    const uint32_t none = ordered(-INFINITY) >> LAST << LAST;
    auto key = [&](int g) { return ordered(most(g)) >> LAST << LAST; };
    uint32_t bound;
    int want;
    bool exact;
    const bool enough = reach<LAST>(B, A.top, [&](auto&& f) {
        for (int i = threadIdx.x; i < G; i += LP_JOIN) {
            const uint32_t k = key(i);
            if (k > none) f(k);
        }
    }, bound, want, exact);
    if (!enough) bound = none + 1;
    if (threadIdx.x == 0) B.chosen = B.found = 0;
    __syncthreads();
    // (in any order: they are only looked through)
    for (int i = threadIdx.x; i < G; i += LP_JOIN) {
        const uint32_t k = key(i);
        if (k > none && (k > bound || (k == bound && (exact || !enough)))) B.group[atomicAdd(&B.chosen, 1)] = i;
    }
    __syncthreads();
    if (!exact && enough && warp == 0) {  // equal ones: the first
        int chosen = B.chosen, left = want;
        for (int i0 = 0; i0 < G && left > 0; i0 += 32) {
            const bool is = i0 + lane < G && key(i0 + lane) == bound;
            const unsigned at = __ballot_sync(0xffffffffu, is), below = (1u << lane) - 1u;
            const int r = __popc(at & below);
            if (is && r < left) B.group[chosen + r] = i0 + lane;
            const int n = min(left, __popc(at));
            chosen += n;
            left -= n;
        }
        if (lane == 0) B.chosen = chosen;
    }
    __syncthreads();
    float least = float_of(bound);
    auto look = [&]() {
        of_groups<DT>(A, row, B, least, [&](float v, int i) {
            const int n = atomicAdd(&B.found, 1);
            if (n < LP_CANDIDATES) {
                B.value[n] = v;
                B.id[n] = i;
            }
        });
        __syncthreads();
        return B.found;
    };
    int found = look();
    if (found > LP_SOME) {
        // few groups, or many as good as the worst group's largest (a small vocabulary): the bound that `top`
        // of the tokens themselves reach
        __syncthreads();
        const float at = least;
        if (reach<LAST>(B, A.top, [&](auto&& f) {
                of_groups<DT>(A, row, B, at, [&](float v, int) { f(ordered(v) >> LAST << LAST); });
            }, bound, want, exact)) {
            least = float_of(bound);
            if (threadIdx.x == 0) B.found = 0;
            __syncthreads();
            found = look();
        }
    }
    int32_t* ids = A.ids + e * A.top;
    float* lps = A.top_lp + e * A.top;
    for (int i = min(found, A.top) + threadIdx.x; i < A.top; i += LP_JOIN) {
        ids[i] = -1;
        lps[i] = -INFINITY;
    }
    if (found <= LP_CANDIDATES) {
        for (int i = threadIdx.x; i < found; i += LP_JOIN) {
            const float v = B.value[i];
            const int id = B.id[i];
            int r = 0;
            for (int j = 0; j < found; ++j) r += before(B.value[j], B.id[j], v, id);
            if (r < A.top) {
                ids[r] = id;
                lps[r] = log_p(v, s, log_z, T);
            }
        }
        return;
    }
    // Many equal ones (a row that is flat at the top): one after another, each the best of
    // what comes after the last.
    float last_v = INFINITY;
    int last_i = -1;
    for (int r = 0; r < A.top; ++r) {
        float v = -INFINITY;
        int id = 0x7fffffff;
        of_groups<DT>(A, row, B, least, [&](float w, int j) {
            if (before(last_v, last_i, w, j) && before(w, j, v, id)) {
                v = w;
                id = j;
            }
        });
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float w = __shfl_xor_sync(0xffffffffu, v, o);
            const int j = __shfl_xor_sync(0xffffffffu, id, o);
            if (before(w, j, v, id)) {
                v = w;
                id = j;
            }
        }
        if (lane == 0) {
            B.round_value[warp] = v;
            B.round_id[warp] = id;
        }
        __syncthreads();
        for (int w = 0; w < LP_JOIN_WARPS; ++w)
            if (before(B.round_value[w], B.round_id[w], v, id)) {
                v = B.round_value[w];
                id = B.round_id[w];
            }
        last_v = v;
        last_i = id;
        if (threadIdx.x == 0) {
            ids[r] = id;
            lps[r] = log_p(v, s, log_z, T);
        }
        __syncthreads();
    }
}

// An entry: its row (-1: nothing is read), kappa = log2(e) / T, and what it reports.
struct Entry {
    long long row;
    int token, bits;
    float kappa, T;
};
__device__ __forceinline__ Entry entry_of(const LogprobArgs& A, long long e) {
    Entry x = {A.rows ? (long long)A.rows[e] : e, A.tokens[e], 0, 1.4426950408889634f, 1.f};
    const float T = A.temp ? A.temp[e] : 0.f;
    if (x.token < 0) {
        x.row = -1;
        return x;
    }
    if (x.token >= A.V || x.row < 0 || x.row >= A.R) x.bits |= int(SPEC_BADBIT_TOKEN);
    if (!(T >= 0.f) || T == INFINITY) x.bits |= int(SPEC_BADBIT_TEMPERATURE);
    if (x.bits) x.row = -1;
    if (T > 0.f) {
        x.kappa = kappa_of(T);
        x.T = T;
    }
    return x;
}
__device__ __forceinline__ void left_out(const LogprobArgs& A, long long e, int bits) {
    if (threadIdx.x == 0) {
        A.lp[e] = 0.f;
        if (A.entropy) A.entropy[e] = 0.f;
        if (bits && A.status) atomicOr(A.status, bits);
    }
    for (int i = threadIdx.x; i < A.top; i += LP_JOIN) {
        A.ids[e * A.top + i] = -1;
        A.top_lp[e * A.top + i] = 0.f;
    }
}
// (one thread)
__device__ __forceinline__ void put_entry(const LogprobArgs& A, float given, const Entry& x, const Sums& s, long long e) {
    const float log_z = log2f(s.z);
    const bool empty = s.z == 0.f;
    A.lp[e] = empty ? -INFINITY : log_p(given, s, log_z, x.T);
    if (A.entropy) A.entropy[e] = empty ? 0.f : 0.6931471805599453f * (log_z - s.a / s.z);
    if (empty && A.status) atomicOr(A.status, int(SPEC_BADBIT_EMPTY_ROW));
}

template <int DT, bool ENT, bool TOP>
__global__ void __launch_bounds__(LP_THREADS, LP_CTAS) k_logprob(const __grid_constant__ LogprobArgs A) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[LP_WARPS][LP_STAGES];
    __shared__ int counts[LP_WARPS];
    __shared__ int32_t near_list[LP_THREADS];  // of few entries
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) {
        for (int i = 0; i < LP_STAGES; ++i) mbar_init(&bars[warp][i], 1);
        fence_mbarrier_init();
    }
    begin_after_previous();

    // The entries that are read: how many, and the list of this CTA's (which it writes for itself).
    auto live = [&](long long e) { return e < A.E && entry_of(A, e).row >= 0; };
    long long total = 0;
    const bool first = live(threadIdx.x);
    int32_t* list = A.E <= LP_THREADS ? near_list : A.list;
    for (long long e0 = 0; e0 < A.E; e0 += LP_THREADS) total += __syncthreads_count(e0 ? live(e0 + threadIdx.x) : first);
    const long long tiles = total * A.tiles, W = (long long)gridDim.x * LP_WARPS;
    // shares of at least one tile: the first CTAs have the work where there is little, a warp each
    const long long w = (long long)warp * gridDim.x + blockIdx.x;
    const bool few = tiles <= W;
    const long long mine = few ? w : (long long)blockIdx.x * LP_WARPS + warp;
    const long long t0 = few ? min(w, tiles) : tiles * mine / W, t1 = few ? min(w + 1, tiles) : tiles * (mine + 1) / W;
    const long long c0 = few ? 0 : tiles * (blockIdx.x * (long long)LP_WARPS) / W, c1 = few ? tiles : tiles * ((blockIdx.x + 1ll) * LP_WARPS) / W;
    const long long a0 = c0 / A.tiles, a1 = (c1 + A.tiles - 1) / A.tiles;  // live entries of the CTA's
    long long before = 0;
    for (long long e0 = 0; e0 < A.E && before < a1; e0 += LP_THREADS) {
        const bool on = e0 ? live(e0 + threadIdx.x) : first;
        const unsigned b = __ballot_sync(0xffffffffu, on);
        if (lane == 0) counts[warp] = __popc(b);
        __syncthreads();
        long long at = before + __popc(b & ((1u << lane) - 1u));
        int all = 0;
#pragma unroll
        for (int i = 0; i < LP_WARPS; ++i) {
            if (i < warp) at += counts[i];
            all += counts[i];
        }
        if (on && at >= a0 && at < a1) list[at] = int32_t(e0 + threadIdx.x);  // (the same by every CTA that writes it)
        before += all;
        __syncthreads();
    }
    if (t0 >= t1) return;

    uint8_t* buf = smem + size_t(warp) * LP_STAGES * LP_BYTES;
    uint64_t* bar = bars[warp];
    // lane 0: the copies
    long long pa = t0 / A.tiles;
    int pc = int(t0 - pa * A.tiles);
    auto bytes_of = [&](const Row<DT>& r, int c) { return uint32_t(max(0, min(LP_VECS, r.vecs - c * LP_VECS))) * 16u; };
    Row<DT> prow(A, entry_of(A, list[pa]).row);
    uint32_t begun = 0;
    long long left = t1 - t0;
    auto issue = [&]() {
        if (left == 0) return;
        const uint32_t st = begun % LP_STAGES, n = bytes_of(prow, pc);
        mbar_arrive_expect_tx(&bar[st], n);
        if (n) bulk_g2s(buf + st * LP_BYTES, reinterpret_cast<const char*>(prow.p + prow.head) + size_t(pc) * LP_BYTES, n, &bar[st]);
        ++begun;
        if (--left && ++pc == A.tiles) {
            pc = 0;
            prow = Row<DT>(A, entry_of(A, list[++pa]).row);
        }
    };
    if (lane == 0)
        for (int i = 0; i < LP_STAGES; ++i) issue();
    long long a = t0 / A.tiles;
    int c = int(t0 - a * A.tiles);
    long long e = list[a];
    Entry x = entry_of(A, e);
    Row<DT> row(A, x.row);
    uint32_t used = 0;
    bool lost = false;
    for (long long t = t0; t < t1; ++t, ++used) {
        const uint32_t st = used % LP_STAGES;
        lost = !__all_sync(0xffffffffu, mbar_wait_bounded(&bar[st], (used / LP_STAGES) & 1u));
        if (lost) break;
        const int vecs = min(LP_VECS, row.vecs - c * LP_VECS);
        const uint4* v = reinterpret_cast<const uint4*>(buf + st * LP_BYTES);
        const uint4 none = make_uint4(Elem<DT>::NONE, Elem<DT>::NONE, Elem<DT>::NONE, Elem<DT>::NONE);
        uint4 d[8];
        if (vecs == LP_VECS) {
#pragma unroll
            for (int k = 0; k < 8; ++k) d[k] = v[k * 32 + lane];
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) d[k] = k * 32 + lane < vecs ? v[k * 32 + lane] : none;
        }
        __syncwarp();  // every lane holds its share: the stage can be filled again
        if (lane == 0) {
            fence_proxy_async_smem();
            issue();
        }
        float mx[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = largest<DT>(d[2 * k], d[2 * k + 1]);
        Lane<DT, ENT> L;
        L.s.m = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), LP_LOWEST);
#pragma unroll
        for (int k = 0; k < 4; ++k) L.take(d[2 * k], d[2 * k + 1], x.kappa);
        if (TOP) {
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = redux_max_f32(mx[k]);
        }
        const Sums s = warp_join<ENT>(L.s, x.kappa);
        if (lane == 0 && vecs > 0) {
            A.part[e * (A.tiles + 1) + c] = make_float4(s.m, s.z, s.a, 0.f);
            if (TOP) A.most[e * (A.tiles + 1) + c] = make_float4(mx[0], mx[1], mx[2], mx[3]);
        }
        if (c == 0) {  // the ends
            const int end = row.end_of(lane);
            const float l = end >= 0 ? to_f32(row.p[end]) : -INFINITY;
            Lane<DT, ENT> K;
            K.one(l, x.kappa);
            const float h = redux_max_f32(lane < 16 ? l : -INFINITY), g = redux_max_f32(lane < 16 ? -INFINITY : l);
            const Sums y = warp_join<ENT>(K.s, x.kappa);
            if (lane == 0) {
                A.part[e * (A.tiles + 1) + A.tiles] = make_float4(y.m, y.z, y.a, 0.f);
                if (TOP) A.most[e * (A.tiles + 1) + A.tiles] = make_float4(h, g, 0.f, 0.f);
            }
        }
        if (++c == A.tiles && t + 1 < t1) {
            c = 0;
            e = list[++a];
            x = entry_of(A, e);
            row = Row<DT>(A, x.row);
        }
    }
    if (lost) {
        if (lane == 0) {
            if (A.status) atomicOr(A.status, int(SPEC_BADBIT_TIMEOUT));
            // copies in flight land before the shared memory is another's
            for (uint32_t i = used; i != begun; ++i) mbar_wait_bounded(&bar[i % LP_STAGES], (i / LP_STAGES) & 1u, 100000000ull);
        }
    }
}

// One CTA an entry: the sums of its row's tiles, and the alternatives.
template <int DT>
__global__ void __launch_bounds__(LP_JOIN) k_logprob_join(const __grid_constant__ LogprobArgs A) {
    begin_after_previous();
    __shared__ Best B;
    constexpr int ROOM = 1280;  // (longer rows' groups are read where they lie)
    __shared__ float kept[ROOM];
    __shared__ float3 parts[LP_JOIN_WARPS];
    const long long e = blockIdx.x;
    const float4* part = A.part + e * (A.tiles + 1);
    const float4* most4 = A.most + e * (A.tiles + 1);
    // (on their way before it is known whether they are used)
    const int early = min(int(threadIdx.x), A.tiles);
    const float4 part0 = __ldcg(part + early), most0 = A.top ? __ldcg(most4 + early) : part0;
    const float4 part_end = __ldcg(part + A.tiles), most_end = A.top ? __ldcg(most4 + A.tiles) : part0;
    const Entry x = entry_of(A, e);
    if (x.row < 0) {
        left_out(A, e, x.bits);
        return;
    }
    const Row<DT> row(A, x.row);
    const float given = to_f32(row.p[x.token]);  // (on its way with the rest)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // groups in the order of their tokens: head, the tiles', tail
    const int G = row.tiles * 4 + 2;
    const bool fits = A.top && G <= ROOM;
    Sums s = {LP_LOWEST, 0.f, 0.f};
    for (int i = threadIdx.x; i <= row.tiles; i += LP_JOIN) {
        const bool end = i == row.tiles, mine = i == int(threadIdx.x);
        const float4 p = end ? part_end : mine ? part0 : __ldcg(part + i);
        if (fits) {
            const float4 m = end ? most_end : mine ? most0 : __ldcg(most4 + i);
            if (i < row.tiles) {
                kept[1 + 4 * i] = m.x;
                kept[2 + 4 * i] = m.y;
                kept[3 + 4 * i] = m.z;
                kept[4 + 4 * i] = m.w;
            } else {
                kept[0] = m.x;
                kept[G - 1] = m.y;
            }
        }
        Sums y = {p.x, p.y, p.z};
        const float m = fmaxf(s.m, y.m);
        s.to(m, x.kappa);
        y.to(m, x.kappa);
        s.z += y.z;
        s.a += y.a;
    }
    s = warp_join<true>(s, x.kappa);
    if (lane == 0) parts[warp] = make_float3(s.m, s.z, s.a);
    __syncthreads();
    const float3 p = lane < LP_JOIN_WARPS ? parts[lane] : make_float3(LP_LOWEST, 0.f, 0.f);
    s = warp_join<true>(Sums{p.x, p.y, p.z}, x.kappa);
    if (threadIdx.x == 0) put_entry(A, given, x, s, e);
    if (!A.top) return;
    auto most = [&](int g) {
        if (fits) return kept[g];
        const float* m = reinterpret_cast<const float*>(most4);
        return __ldcg(g == 0 ? m + 4 * A.tiles : g == G - 1 ? m + 4 * A.tiles + 1 : m + g - 1);
    };
    best_tokens<DT>(A, row, B, most, s, x.T, e);
}

template <int DT>
cudaError_t launch_logprob(const LogprobArgs& A, int sms, cudaStream_t st) {
    auto* kernel = A.entropy ? (A.top ? k_logprob<DT, true, true> : k_logprob<DT, true, false>)
                             : (A.top ? k_logprob<DT, false, true> : k_logprob<DT, false, false>);
    static bool ready[64][4] = {};  // per device; setting it twice does no harm
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    bool& set = ready[dev][(A.entropy ? 2 : 0) + (A.top ? 1 : 0)];
    if (!set) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(LP_SMEM));
        if (e != cudaSuccess) return e;
        set = true;
    }
    e = launch_behind(kernel, dim3(unsigned(std::min<long long>((long long)LP_CTAS * sms, A.E * A.tiles))), LP_THREADS, LP_SMEM, st, A);
    if (e != cudaSuccess) return e;
    return launch_behind(k_logprob_join<DT>, dim3(unsigned(A.E)), LP_JOIN, 0, st, A);
}

// tiles of a row, at most
int tiles_of(int V, int bytes) { return std::max(1, (V / (16 / bytes) + LP_VECS - 1) / LP_VECS); }
size_t list_bytes(long long E) { return align256(size_t(E) * 4); }
size_t part_bytes(long long E, int tiles) { return align256(size_t(E) * (tiles + 1) * sizeof(float4)); }

constexpr long long LP_MAX_ENTRIES = 1 << 24;

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

size_t spec_token_logprobs_workspace_size(int64_t E, int V) {
    if (E < 0 || E > LP_MAX_ENTRIES || V < 1 || V > (1 << 24)) return 0;
    const int tiles = tiles_of(V, 4);  // (the element's size is not known here: the larger)
    return list_bytes(E) + 2 * part_bytes(E, tiles) + 256;
}

spec_status spec_token_logprobs(const void* logits, spec_dtype dtype, int64_t R, int64_t row_stride, int V, const int32_t* rows,
                                const int32_t* tokens, const float* temperature, int64_t E, int top, float* logprobs,
                                float* entropy, int32_t* top_ids, float* top_logprobs, void* workspace,
                                size_t workspace_bytes, int32_t* dev_status, spec_stream_t stream) {
    if (R < 0 || E < 0 || V < 1 || top < 0 || top > SPEC_MAX_TOP || (!rows && E > R)) return SPEC_ERR_INVALID_ARG;
    if (dtype != SPEC_F32 && dtype != SPEC_BF16 && dtype != SPEC_F16) return SPEC_ERR_INVALID_ARG;
    if (R > 1 && row_stride < V) return SPEC_ERR_INVALID_ARG;
    if (V > (1 << 24) || E > LP_MAX_ENTRIES || R > (1ll << 31) || row_stride > (1ll << 38)) return SPEC_ERR_UNSUPPORTED;
    if (E == 0) return SPEC_OK;
    if ((R && !logits) || !tokens || !logprobs || (top && (!top_ids || !top_logprobs)) || !workspace)
        return SPEC_ERR_INVALID_ARG;
    if (!aligned(logits, dtype_bytes(dtype)) ||
        !all_aligned(4, {rows, tokens, temperature, logprobs, entropy, top_ids, top_logprobs, dev_status}))
        return SPEC_ERR_UNSUPPORTED;
    const int sms = sm_count();
    if (sms <= 0) return SPEC_ERR_CUDA;
    if (!aligned(workspace, 256) || workspace_bytes < spec_token_logprobs_workspace_size(E, V)) return SPEC_ERR_WORKSPACE;
    LogprobArgs A = {};
    A.logits = logits;
    A.R = R;
    A.stride = row_stride;
    A.rows = rows;
    A.tokens = tokens;
    A.temp = temperature;
    A.lp = logprobs;
    A.entropy = entropy;
    A.ids = top_ids;
    A.top_lp = top_logprobs;
    A.tiles = tiles_of(V, dtype_bytes(dtype));
    char* room = static_cast<char*>(workspace);
    A.list = reinterpret_cast<int32_t*>(room);
    A.part = reinterpret_cast<float4*>(room += list_bytes(E));
    A.most = reinterpret_cast<float4*>(room + part_bytes(E, A.tiles));
    A.status = dev_status;
    A.V = V;
    A.top = top;
    A.E = E;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == SPEC_F32    ? launch_logprob<SPEC_F32>(A, sms, st)
                          : dtype == SPEC_BF16 ? launch_logprob<SPEC_BF16>(A, sms, st)
                                               : launch_logprob<SPEC_F16>(A, sms, st);
    return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"
