// logprob.cu -- spec_token_logprobs: log probabilities of given tokens, the entropy of
// their distributions and the most probable alternatives, each row of logits read once.
//
// With M the largest logit, a(x) = (l(x) - M) log2(e) / T, Z = sum 2^a, and A = sum 2^a a:
//   log p(x) = (l(x) - M) / T - ln 2 log2 Z,   H = ln 2 (log2 Z - A / Z).
// Each lane keeps (M, Z, A) of what it has seen, by a maximum of its own; a larger one turns
// (Z, A) into f Z, f (A + d Z), f = 2^d, d the difference, and so do the joins of lanes,
// warps and CTAs.
//
// Alternatives.  A row is cut into groups of 512 neighbours (256 of f32; of long rows several of
// those), and the pass leaves each group's largest logit behind.  The k best tokens lie
// in the k groups whose largest are best (by value, then by place: each of those k is itself a
// token, and no other group's is as good), so that the k groups alone are read a second
// time, out of L2, for tokens as good as the k-th group's largest.
//
// k_logprob takes a row with one CTA where there are two rows an SM and more, else
// several share a row, and k_logprob_join, launched behind it, joins their sums.
// Bound by HBM for many rows; by latency for few.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "cache.cuh"

namespace sv {
namespace {

constexpr int LP_THREADS = 512, LP_WARPS = LP_THREADS / 32;
constexpr int LP_GROUPS = 1024;  // groups of a row between its ends, at most
constexpr int LP_CANDIDATES = 1024;
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
    float4* part;  // [E][splits] {M, Z, A}
    float* most;   // [E][groups + 2] largest logits, where several CTAs share a row
    int32_t* status;
    int V, top, splits, span;  // span: units of a group
    int groups;                // of a row between its ends, at most
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
    int head, vecs, units, groups, tail;
    __device__ __forceinline__ Row(const LogprobArgs& A, long long row) {
        p = static_cast<const T*>(A.logits) + row * A.stride;
        head = min(A.V, int((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / Elem<DT>::SIZE);
        vecs = (A.V - head) / Elem<DT>::EPV;
        tail = A.V - head - vecs * Elem<DT>::EPV;
        units = (vecs + 63) / 64;
        groups = (units + A.span - 1) / A.span;
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
    __device__ __forceinline__ void take(const uint4& u, const uint4& v, float mx, float kappa) {
        s.to(fmaxf(s.m, mx), kappa);
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
__device__ __forceinline__ Sums warp_join(Sums s, float kappa) {
    s.to(redux_max_f32(s.m), kappa);
    s.z = warp_sum_f(s.z);
    s.a = warp_sum_f(s.a);
    return s;
}

// (by the temperature itself: the difference from a logit that a mask made the lowest float
// would not be one any more in units of log2(e) / T)
__device__ __forceinline__ float log_p(float l, const Sums& s, float log_z, float T) {
    return (l - s.m) / T - 0.6931471805599453f * log_z;
}

struct Best {  // what a CTA needs for the alternatives
    float most[LP_GROUPS + 2];
    float value[LP_CANDIDATES];
    int id[LP_CANDIDATES];
    int group[SPEC_MAX_TOP];
    float at_least;
    int chosen, found;
    float round_value[LP_WARPS];
    int round_id[LP_WARPS];
};

// largest first, of equal ones the lowest index
__device__ __forceinline__ bool before(float v, int i, float w, int j) { return v > w || (v == w && i < j); }
__device__ __forceinline__ uint32_t ordered(float f) {  // (0 and -0 alike)
    const uint32_t u = __float_as_uint(f + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// f(value, index) for every element of a chosen group, by the warps of the CTA in turn
template <int DT, class F>
__device__ __forceinline__ void of_groups(const LogprobArgs& A, const Row<DT>& row, const Best& B, F&& f) {
    constexpr int EPV = Elem<DT>::EPV;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int c = warp; c < B.chosen; c += LP_WARPS) {
        const int g = B.group[c] - 1;
        if (g < 0 || g >= row.groups) {
            const int e = row.end_of(lane);
            if (e >= 0 && (lane < 16) == (g < 0)) f(to_f32(row.p[e]), e);
            continue;
        }
        for (int u = g * A.span; u < min(row.units, (g + 1) * A.span); ++u)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int i = u * 64 + y * 32 + lane;
                float x[EPV];
                unpack<DT>(row.vec(i), x);
                if (i < row.vecs)
#pragma unroll
                    for (int e = 0; e < EPV; ++e) f(x[e], row.head + i * EPV + e);
            }
    }
}

// The alternatives of a row whose groups' largest logits lie in B.most (all of the CTA).
template <int DT>
__device__ __forceinline__ void best_tokens(const LogprobArgs& A, const Row<DT>& row, Best& B, const Sums& s, float T,
                                            long long e) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = row.groups + 2;
    const float log_z = log2f(s.z);
    if (warp == 0) {
        // the largest bound that `top` groups reach, bit by bit; those above it, and of
        // those at it the first
        auto reach = [&](uint32_t bound) {
            int n = 0;
            for (int i = lane; i < G; i += 32) n += ordered(B.most[i]) >= bound;
            return int(__reduce_add_sync(0xffffffffu, unsigned(n)));
        };
        const uint32_t none = ordered(-INFINITY);
        uint32_t bound = none + 1;
        if (reach(bound) > A.top) {
            uint32_t at = 0;
            for (int bit = 31; bit >= 0; --bit) {
                const uint32_t t = at | 1u << bit;
                const int n = t > none ? reach(t) : A.top;
                if (n >= A.top) at = t;
                if (n == A.top && t > none) break;
            }
            bound = max(at, none + 1);
        }
        int chosen = 0, left = A.top - reach(bound + 1);
        for (int i0 = 0; i0 < G; i0 += 32) {
            const uint32_t k = i0 + lane < G ? ordered(B.most[i0 + lane]) : 0u;
            const unsigned at = __ballot_sync(0xffffffffu, k == bound), below = (1u << lane) - 1u;
            const bool take = k > bound || (k == bound && __popc(at & below) < left);
            left -= min(left, __popc(at));
            const unsigned all = __ballot_sync(0xffffffffu, take);
            if (take) B.group[chosen + __popc(all & below)] = i0 + lane;
            chosen += __popc(all);
        }
        if (lane == 0) {
            B.chosen = chosen;
            B.found = 0;
            const uint32_t u = bound;
            B.at_least = __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
        }
    }
    __syncthreads();
    const float bound = B.at_least;
    of_groups<DT>(A, row, B, [&](float v, int i) {
        if (v >= bound) {
            const int n = atomicAdd(&B.found, 1);
            if (n < LP_CANDIDATES) {
                B.value[n] = v;
                B.id[n] = i;
            }
        }
    });
    __syncthreads();
    const int found = B.found;
    int32_t* ids = A.ids + e * A.top;
    float* lps = A.top_lp + e * A.top;
    for (int i = min(found, A.top) + threadIdx.x; i < A.top; i += LP_THREADS) {
        ids[i] = -1;
        lps[i] = -INFINITY;
    }
    if (found <= LP_CANDIDATES) {
        for (int i = threadIdx.x; i < found; i += LP_THREADS) {
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
        of_groups<DT>(A, row, B, [&](float w, int j) {
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
        for (int w = 0; w < LP_WARPS; ++w)
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
    for (int i = threadIdx.x; i < A.top; i += LP_THREADS) {
        A.ids[e * A.top + i] = -1;
        A.top_lp[e * A.top + i] = 0.f;
    }
}
// (one thread)
template <int DT>
__device__ __forceinline__ void put_entry(const LogprobArgs& A, const Row<DT>& row, const Entry& x, const Sums& s, long long e) {
    const float log_z = log2f(s.z);
    const bool empty = s.z == 0.f;
    A.lp[e] = empty ? -INFINITY : log_p(to_f32(row.p[x.token]), s, log_z, x.T);
    if (A.entropy) A.entropy[e] = empty ? 0.f : 0.6931471805599453f * (log_z - s.a / s.z);
    if (empty && A.status) atomicOr(A.status, int(SPEC_BADBIT_EMPTY_ROW));
}

template <int DT, bool ENT, bool TOP>
__global__ void __launch_bounds__(LP_THREADS, 2) k_logprob(const __grid_constant__ LogprobArgs A) {
    begin_after_previous();
    __shared__ Best B;
    __shared__ float3 parts[LP_WARPS];
    const long long e = blockIdx.x / unsigned(A.splits);
    const int split = int(blockIdx.x - unsigned(e) * unsigned(A.splits));
    const Entry x = entry_of(A, e);
    const bool alone = A.splits == 1;
    if (x.row < 0) {
        if (alone) left_out(A, e, x.bits);
        return;
    }
    const Row<DT> row(A, x.row);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* most = alone ? B.most : A.most + e * (A.groups + 2);
    const int g0 = int((long long)row.groups * split / A.splits), g1 = int((long long)row.groups * (split + 1) / A.splits);
    Lane<DT, ENT> L;
    // a group's units, the next one's loads under way while one is worked on
    int g = g0 + warp, u = g * A.span;
    uint4 a, b;
    auto load = [&](int u) {
        a = row.vec(u * 64 + lane);
        b = row.vec(u * 64 + 32 + lane);
    };
    if (g < g1) load(u);
    float in_group = -INFINITY;
    while (g < g1) {
        const uint4 va = a, vb = b;
        const int of = g;
        bool done = false;
        if (++u == (g + 1) * A.span || u >= row.units) {
            g += LP_WARPS;
            u = g * A.span;
            done = true;
        }
        if (g < g1) load(u);
        const float mx = largest<DT>(va, vb);
        in_group = fmaxf(in_group, mx);
        L.take(va, vb, mx, x.kappa);
        if (TOP && done) {
            const float all = redux_max_f32(in_group);
            if (lane == 0) most[of + 1] = all;
            in_group = -INFINITY;
        }
    }
    if (split == 0 && warp == LP_WARPS - 1) {  // the ends
        const int end = row.end_of(lane);
        const float l = end >= 0 ? to_f32(row.p[end]) : -INFINITY;
        L.one(l, x.kappa);
        if (TOP) {
            const float h = redux_max_f32(lane < 16 ? l : -INFINITY), t = redux_max_f32(lane < 16 ? -INFINITY : l);
            if (lane == 0) {
                most[0] = h;
                most[row.groups + 1] = t;
            }
        }
    }
    Sums s = warp_join(L.s, x.kappa);
    if (lane == 0) parts[warp] = make_float3(s.m, s.z, s.a);
    __syncthreads();
    if (alone && TOP) {  // every warp needs the sums
        const float3 p = lane < LP_WARPS ? parts[lane] : make_float3(LP_LOWEST, 0.f, 0.f);
        s = warp_join(Sums{p.x, p.y, p.z}, x.kappa);
        if (threadIdx.x == 0) put_entry<DT>(A, row, x, s, e);
        best_tokens<DT>(A, row, B, s, x.T, e);
    } else if (warp == 0) {
        const float3 p = lane < LP_WARPS ? parts[lane] : make_float3(LP_LOWEST, 0.f, 0.f);
        s = warp_join(Sums{p.x, p.y, p.z}, x.kappa);
        if (lane == 0) {
            if (alone) put_entry<DT>(A, row, x, s, e);
            else A.part[e * A.splits + split] = make_float4(s.m, s.z, s.a, 0.f);
        }
    }
}

// One CTA an entry: the sums of its row's CTAs, and the alternatives.
template <int DT>
__global__ void __launch_bounds__(LP_THREADS) k_logprob_join(const __grid_constant__ LogprobArgs A) {
    begin_after_previous();
    __shared__ Best B;
    const long long e = blockIdx.x;
    const Entry x = entry_of(A, e);
    if (x.row < 0) {
        left_out(A, e, x.bits);
        return;
    }
    const Row<DT> row(A, x.row);
    const int lane = threadIdx.x & 31;
    if (A.top)
        for (int i = threadIdx.x; i < row.groups + 2; i += LP_THREADS) B.most[i] = __ldcg(A.most + e * (A.groups + 2) + i);
    Sums s = {LP_LOWEST, 0.f, 0.f};
    for (int i = lane; i < A.splits; i += 32) {
        const float4 p = __ldcg(A.part + e * A.splits + i);
        Sums y = {p.x, p.y, p.z};
        const float m = fmaxf(s.m, y.m);
        s.to(m, x.kappa);
        y.to(m, x.kappa);
        s.z += y.z;
        s.a += y.a;
    }
    s = warp_join(s, x.kappa);
    if (threadIdx.x == 0) put_entry<DT>(A, row, x, s, e);
    if (!A.top) return;
    __syncthreads();
    best_tokens<DT>(A, row, B, s, x.T, e);
}

template <int DT>
cudaError_t launch_logprob(const LogprobArgs& A, long long E, cudaStream_t st) {
    auto* kernel = A.entropy ? (A.top ? k_logprob<DT, true, true> : k_logprob<DT, true, false>)
                             : (A.top ? k_logprob<DT, false, true> : k_logprob<DT, false, false>);
    const cudaError_t e = launch_behind(kernel, dim3(unsigned(E * A.splits)), LP_THREADS, 0, st, A);
    if (e != cudaSuccess || A.splits == 1) return e;
    return launch_behind(k_logprob_join<DT>, dim3(unsigned(E)), LP_THREADS, 0, st, A);
}

// elements that a warp takes at once: two vectors a lane
constexpr int unit_of(int bytes) { return 64 * 16 / bytes; }
// How a call of E entries and V tokens is cut.
// A row takes one CTA from two rows an SM on (an SM holds two CTAs), else as many as fill the
// GPU twice, with a group a warp at least.
struct Cut {
    int span, groups, splits;
};
Cut cut_of(long long E, int V, int unit, int sms) {
    Cut c;
    const int units = (V + unit - 1) / unit;
    c.span = (units + LP_GROUPS - 1) / LP_GROUPS;
    c.groups = (units + c.span - 1) / c.span;
    const long long want = (2ll * sms + E - 1) / E;
    c.splits = int(std::max(1ll, std::min(want, (long long)(c.groups + LP_WARPS - 1) / LP_WARPS)));
    return c;
}
size_t part_bytes(long long E, const Cut& c) { return align256(size_t(E) * c.splits * sizeof(float4)); }
size_t most_bytes(long long E, const Cut& c) { return align256(size_t(E) * (c.groups + 2) * 4); }

constexpr long long LP_MAX_ENTRIES = 1 << 24;

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

size_t spec_token_logprobs_workspace_size(int64_t E, int V) {
    if (E < 0 || E > LP_MAX_ENTRIES || V < 1 || V > (1 << 24)) return 0;
    const int sms = sm_count();
    if (sms <= 0) return 0;
    if (E == 0) return 256;
    size_t n = 256;  // (the element's size is not known here)
    for (int bytes : {4, 2}) {
        const Cut c = cut_of(E, V, unit_of(bytes), sms);
        if (c.splits > 1) n = std::max(n, part_bytes(E, c) + most_bytes(E, c));
    }
    return n;
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
    const Cut c = cut_of(E, V, unit_of(dtype_bytes(dtype)), sms);
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
    A.part = static_cast<float4*>(workspace);
    A.most = reinterpret_cast<float*>(static_cast<char*>(workspace) + part_bytes(E, c));
    A.status = dev_status;
    A.V = V;
    A.top = top;
    A.splits = c.splits;
    A.span = c.span;
    A.groups = c.groups;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == SPEC_F32    ? launch_logprob<SPEC_F32>(A, E, st)
                          : dtype == SPEC_BF16 ? launch_logprob<SPEC_BF16>(A, E, st)
                                               : launch_logprob<SPEC_F16>(A, E, st);
    return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"
