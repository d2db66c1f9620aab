// rope.cu -- rotary positions, and the cache rows written and read.
//
// k_rotate turns the heads of a token by its position's angles and stores
// them: to a tensor (spec_rope), or to the token's cache slot, as they are or
// in 8 bits (spec_kv_write).  A group of GS lanes takes one token and a share
// of its heads; lane i of the group keeps item i of each head:
//   an item of the rotated part: VEC pairs (half layout: two vectors rot / 2
//     channels apart; interleaved: one vector of VEC / 2 pairs);
//   an item of the rest of the head: one vector, copied.
// So the sines and cosines of an item are computed once for all heads of the
// share, and an e4m3 row's maximum is a shuffle within the group.
//
// The angle.  turns[i] is theta_i / (2 pi) as a fraction of 2^64, so the low
// 64 bits of position * turns[i] are the exact fraction of a turn (two 32-bit
// multiplies give its top half, which is all that float32 can use); sincospif
// of that fraction needs no range reduction.  The float32 product position *
// theta_i would be off by up to 2^-24 of the whole angle: 0.06 radians at a
// position of a million.
//
// The kernels are bound by memory: every byte is read and written once.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "cache.cuh"

namespace sv {

int sm_count() {
    static std::mutex mu;
    static int sms[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lk(mu);
    if (!sms[dev] && cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return sms[dev];
}

namespace {

constexpr int ROT_THREADS = 256;

struct Heads {  // one side of a rotated tensor
    const void* in;
    void* out;
    long long it, ih, ot, oh;  // token and head strides, elements
    int n;
};

struct RotArgs {
    Heads q, k, v;  // v: only with a cache
    const int32_t* pos;
    const unsigned long long* turns;
    int half_rot;  // pairs that turn (0: none)
    int interleaved;
    float scale, sign;
    int D;
    long long T;
    int share;   // heads a group takes
    int shares;  // groups of a token
    // cache (k and v go to the token's slot)
    CacheView c;
    const long long* slots;
    int32_t* status;
};

__device__ __forceinline__ void angle(unsigned long long turns, int pos, float& c, float& s) {
    // bits 63..32 of pos * turns as a signed fraction of a turn, in half turns
    const uint32_t hi = uint32_t(pos) * uint32_t(turns >> 32) +
                        __umulhi(uint32_t(pos), uint32_t(turns)) -
                        (pos < 0 ? uint32_t(turns) : 0u);
    sincospif(float(int32_t(hi)) * 4.656612873077393e-10f, &s, &c);  // 2^-31
}

template <typename T, int N, bool WIDE>
__device__ __forceinline__ Vec<T, N> load_els(const T* p) {
    if constexpr (WIDE) return load_vec<T, N>(p);
    Vec<T, N> v;
#pragma unroll
    for (int e = 0; e < N; ++e) v.e[e] = p[e];
    return v;
}
template <typename T, int N, bool WIDE>
__device__ __forceinline__ void store_els(T* p, const Vec<T, N>& v) {
    if constexpr (WIDE) {
        store_vec<T, N>(p, v);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) p[e] = v.e[e];
    }
}

__device__ __forceinline__ int items_of(int D, int half_rot, int interleaved, int vec) {
    return interleaved || half_rot == 0 ? D / vec : half_rot / vec + (D - 2 * half_rot) / vec;
}

// T: element type of the tensors; VEC: elements of a vector; GS: lanes of a
// group; E4: the cache is e4m3 (else of type T); WIDE: vectors are aligned
// (else they are read and written element by element).
template <typename T, int VEC, int GS, bool E4, bool WIDE>
__global__ void __launch_bounds__(ROT_THREADS) k_rotate(const __grid_constant__ RotArgs A) {
    const int items = items_of(A.D, A.half_rot, A.interleaved, VEC);
    const int lane = threadIdx.x % GS;
    const unsigned gmask = GS == 32 ? 0xffffffffu
                                    : ((1u << GS) - 1u) << (((threadIdx.x & 31) / GS) * GS);
    const long long groups = A.T * A.shares;
    const int H = A.q.n + A.k.n + A.v.n;
    for (long long g = blockIdx.x * (long long)(ROT_THREADS / GS) + threadIdx.x / GS; g < groups;
         g += (long long)gridDim.x * (ROT_THREADS / GS)) {
        const long long t = g / A.shares;
        const int h0 = int(g - t * A.shares) * A.share, h1 = min(H, h0 + A.share);
        const int pos = A.half_rot ? A.pos[t] : 0;
        long long slot = -1, row = 0, srow = 0;
        if (A.slots) {
            slot = A.slots[t];
            if (slot >= A.c.slots) {
                if (lane == 0 && A.status) atomicOr(A.status, int(SPEC_BADBIT_PAGE));
                slot = -1;
            }
            if (slot >= 0) {
                const long long p = slot / A.c.page;
                const int o = int(slot - p * A.c.page);
                row = p * A.c.page_stride + o * A.c.token_stride;
                srow = p * A.c.heads * A.c.page + o;
            }
        }
        // sines and cosines of this lane's (first) item
        float cs[VEC], sn[VEC];
        auto trig = [&](int i) {
            const int n = A.interleaved ? VEC / 2 : VEC, i0 = i * n;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                if (e >= n || i0 + e >= A.half_rot) break;
                float c, s;
                angle(A.turns[i0 + e], pos, c, s);
                cs[e] = c * A.scale;
                sn[e] = s * A.scale * A.sign;
            }
        };
        if (A.half_rot) trig(lane);
        for (int h = h0; h < h1; ++h) {
            const int kind = h < A.q.n ? 0 : h < A.q.n + A.k.n ? 1 : 2;
            const Heads& X = kind == 0 ? A.q : kind == 1 ? A.k : A.v;
            const int hh = kind == 0 ? h : kind == 1 ? h - A.q.n : h - A.q.n - A.k.n;
            const bool cached = A.slots && kind != 0;
            if (cached && slot < 0) continue;
            const bool turn = kind != 2 && A.half_rot;
            // values of a head that does not turn are cut into plain vectors
            const int n_items = turn ? items : A.D / VEC;
            const T* in = static_cast<const T*>(X.in) + t * X.it + hh * X.ih;
            // the rotated values of item i: va (and vb, `second` channels on)
            float va[VEC], vb[VEC];
            auto get = [&](int i, int& off, int& second) {
                off = i * VEC;
                second = 0;
                bool turns = turn && A.interleaved && i * VEC < 2 * A.half_rot;
                if (turn && !A.interleaved) {
                    const int r = A.half_rot / VEC;
                    if (i < r) {
                        second = A.half_rot;
                        turns = true;
                    } else {
                        off = 2 * A.half_rot + (i - r) * VEC;
                    }
                }
                const Vec<T, VEC> x = load_els<T, VEC, WIDE>(in + off);
#pragma unroll
                for (int e = 0; e < VEC; ++e) va[e] = to_f32(x.e[e]);
                if (second) {
                    const Vec<T, VEC> y = load_els<T, VEC, WIDE>(in + off + second);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        vb[e] = to_f32(y.e[e]);
                        const float a = va[e], b = vb[e];
                        va[e] = a * cs[e] - b * sn[e];
                        vb[e] = a * sn[e] + b * cs[e];
                    }
                } else if (turns) {
#pragma unroll
                    for (int e = 0; e < VEC / 2; ++e) {
                        const float a = va[2 * e], b = va[2 * e + 1];
                        va[2 * e] = a * cs[e] - b * sn[e];
                        va[2 * e + 1] = a * sn[e] + b * cs[e];
                    }
                }
            };
            if (E4 && cached) {
                float amax = 0.f;
                int off = 0, second = 0;
                for (int i = lane; i < n_items; i += GS) {
                    if (turn && i != lane) trig(i);
                    get(i, off, second);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        amax = fmaxf(amax, finite_abs(va[e]));
                        if (second) amax = fmaxf(amax, finite_abs(vb[e]));
                    }
                }
#pragma unroll
                for (int o = GS / 2; o; o >>= 1)
                    amax = fmaxf(amax, __shfl_xor_sync(gmask, amax, o, GS));
                const int ex = e4m3_exponent(amax);
                uint8_t* out = static_cast<uint8_t*>(kind == 1 ? A.c.k : A.c.v) + row +
                               hh * A.c.head_stride;
                for (int i = lane; i < n_items; i += GS) {
                    if (n_items > GS) {  // more than one item: they are made again
                        if (turn) trig(i);
                        get(i, off, second);
                    }
                    auto put = [&](const float (&f)[VEC], int at) {
                        Vec<uint8_t, VEC> o;
                        if constexpr (VEC == 1) {
                            o.e[0] = uint8_t(pack_e4m3x2(e4m3_scaled(f[0], ex), 0.f));
                        } else {
#pragma unroll
                            for (int e = 0; e < VEC; e += 2) {
                                const uint16_t w = pack_e4m3x2(e4m3_scaled(f[e], ex),
                                                               e4m3_scaled(f[e + 1], ex));
                                o.e[e] = uint8_t(w);
                                o.e[e + 1] = uint8_t(w >> 8);
                            }
                        }
                        store_els<uint8_t, VEC, WIDE>(out + at, o);
                    };
                    put(va, off);
                    if (second) put(vb, off + second);
                }
                if (lane == 0)
                    (kind == 1 ? A.c.ks : A.c.vs)[srow + (long long)hh * A.c.page] = uint8_t(ex + 127);
                if (turn && n_items > GS) trig(lane);
            } else {
                T* out = cached ? static_cast<T*>(kind == 1 ? A.c.k : A.c.v) + row + hh * A.c.head_stride
                                : static_cast<T*>(X.out) + t * X.ot + hh * X.oh;
                for (int i = lane; i < n_items; i += GS) {
                    if (turn && i != lane) trig(i);
                    int off, second;
                    get(i, off, second);
                    Vec<T, VEC> o;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) o.e[e] = from_f32<T>(va[e]);
                    store_els<T, VEC, WIDE>(out + off, o);
                    if (second) {
#pragma unroll
                        for (int e = 0; e < VEC; ++e) o.e[e] = from_f32<T>(vb[e]);
                        store_els<T, VEC, WIDE>(out + off + second, o);
                    }
                }
                if (turn && n_items > GS) trig(lane);
            }
        }
    }
}

// Rows of T slots: one thread per 8 channels of a (token, head).
template <typename C, typename T>
__global__ void __launch_bounds__(256) k_kv_read(CacheView c, long long T_, const long long* slots,
                                                 T* out_k, T* out_v) {
    const int vecs = c.D / 8;
    const long long n = T_ * c.heads * vecs;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
        const long long th = i / vecs;
        const int d = int(i - th * vecs) * 8;
        const long long t = th / c.heads;
        const int h = int(th - t * c.heads);
        const long long slot = slots[t];
        Vec<T, 8> ok, ov;
#pragma unroll
        for (int e = 0; e < 8; ++e) ok.e[e] = ov.e[e] = from_f32<T>(0.f);
        if (slot >= 0 && slot < c.slots) {
            const long long p = slot / c.page;
            const int o = int(slot - p * c.page);
            const long long at = p * c.page_stride + h * c.head_stride + o * c.token_stride + d;
            if constexpr (sizeof(C) == 1) {
                const long long sr = (p * c.heads + h) * c.page + o;
                const int ek = int(c.ks[sr]) - 127, ev = int(c.vs[sr]) - 127;
                const Vec<uint16_t, 4> k = load_vec<uint16_t, 4>(
                    reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(c.k) + at));
                const Vec<uint16_t, 4> v = load_vec<uint16_t, 4>(
                    reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(c.v) + at));
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t wk = e4m3x2_to_f16x2(k.e[e]), wv = e4m3x2_to_f16x2(v.e[e]);
                    const float2 fk = __half22float2(*reinterpret_cast<const __half2*>(&wk));
                    const float2 fv = __half22float2(*reinterpret_cast<const __half2*>(&wv));
                    ok.e[2 * e] = from_f32<T>(ldexpf(fk.x, ek));
                    ok.e[2 * e + 1] = from_f32<T>(ldexpf(fk.y, ek));
                    ov.e[2 * e] = from_f32<T>(ldexpf(fv.x, ev));
                    ov.e[2 * e + 1] = from_f32<T>(ldexpf(fv.y, ev));
                }
            } else {
                const Vec<C, 8> k = load_vec<C, 8>(static_cast<const C*>(c.k) + at);
                const Vec<C, 8> v = load_vec<C, 8>(static_cast<const C*>(c.v) + at);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    ok.e[e] = from_f32<T>(to_f32(k.e[e]));
                    ov.e[e] = from_f32<T>(to_f32(v.e[e]));
                }
            }
        }
        store_vec<T, 8>(out_k + i * 8, ok);
        store_vec<T, 8>(out_v + i * 8, ov);
    }
}

template <typename T, int VEC, bool E4, bool WIDE = true>
cudaError_t launch_rotate(RotArgs A, cudaStream_t st) {
    const int rot_items = A.interleaved || !A.half_rot
                              ? A.D / VEC
                              : A.half_rot / VEC + (A.D - 2 * A.half_rot) / VEC;
    // v heads of a call that rotates k are cut into D / VEC vectors
    const int items = A.v.n && !E4 ? rot_items : std::max(rot_items, A.v.n ? A.D / VEC : 0);
    const int gs = items <= 8 ? 8 : items <= 16 ? 16 : 32;
    const int H = A.q.n + A.k.n + A.v.n, sms = sm_count();
    if (sms <= 0) return cudaErrorUnknown;
    // heads a group takes: one while that leaves SMs short of groups, up to 8
    int share = 1;
    while (share < 8 && share < H && A.T * ((H + 2 * share - 1) / (2 * share)) * gs >= 2048ll * sms)
        share *= 2;
    A.share = share;
    A.shares = (H + share - 1) / share;
    const long long groups = A.T * A.shares, per = ROT_THREADS / gs;
    const long long grid = std::min<long long>((groups + per - 1) / per, 1ll << 30);
    if (gs == 8) k_rotate<T, VEC, 8, E4, WIDE><<<unsigned(grid), ROT_THREADS, 0, st>>>(A);
    else if (gs == 16) k_rotate<T, VEC, 16, E4, WIDE><<<unsigned(grid), ROT_THREADS, 0, st>>>(A);
    else k_rotate<T, VEC, 32, E4, WIDE><<<unsigned(grid), ROT_THREADS, 0, st>>>(A);
    return cudaGetLastError();
}

template <typename T, bool E4>
cudaError_t launch_rotate_vec(const RotArgs& A, cudaStream_t st) {
    // the widest vector that every offset of the call is a multiple of: 8
    // elements or 4; else pairs (interleaved) or single elements, one by one
    auto ok = [&](int vec) {
        const size_t a = std::min<size_t>(16, vec * sizeof(T));
        auto side = [&](const Heads& h, bool out) {
            if (!h.n) return true;
            if (!aligned(h.in, a) || h.it % vec || h.ih % vec) return false;
            return !out || (aligned(h.out, a) && h.ot % vec == 0 && h.oh % vec == 0);
        };
        if (A.D % vec || (A.interleaved ? 2 * A.half_rot : A.half_rot) % vec) return false;
        return side(A.q, true) && side(A.k, !A.slots) && side(A.v, false);
    };
    if (ok(8)) return launch_rotate<T, 8, E4>(A, st);
    if (ok(4)) return launch_rotate<T, 4, E4>(A, st);
    if (A.interleaved) return launch_rotate<T, 2, E4, false>(A, st);
    return launch_rotate<T, 1, E4, false>(A, st);
}

spec_status check_table(const spec_rope_table* t, int D) {
    if (!t->turns || t->rot < 2 || t->rot > D || t->rot % 2) return SPEC_ERR_INVALID_ARG;
    if (t->layout != SPEC_ROPE_HALF && t->layout != SPEC_ROPE_INTERLEAVED)
        return SPEC_ERR_INVALID_ARG;
    if (!aligned(t->turns, 8)) return SPEC_ERR_UNSUPPORTED;
    return SPEC_OK;
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

spec_status spec_rope_turns(int rot, double base, int scaling, double factor, double original_len,
                            double fast, double slow, uint64_t* out_turns, float* out_scale) {
    if (!out_turns || !out_scale || rot < 2 || rot > 256 || rot % 2 || !(base > 1.0))
        return SPEC_ERR_INVALID_ARG;
    if (scaling < SPEC_ROPE_PLAIN || scaling > SPEC_ROPE_BY_PARTS) return SPEC_ERR_INVALID_ARG;
    if (scaling != SPEC_ROPE_PLAIN && !(factor >= 1.0)) return SPEC_ERR_INVALID_ARG;
    if (scaling == SPEC_ROPE_BY_PARTS && (!(original_len > 0.0) || !(fast > slow)))
        return SPEC_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925286766559;
    if (scaling == SPEC_ROPE_NTK) base *= std::pow(factor, double(rot) / std::max(1, rot - 2));
    for (int i = 0; i < rot / 2; ++i) {
        double th = std::pow(base, -2.0 * i / rot);
        if (scaling == SPEC_ROPE_LINEAR) th /= factor;
        if (scaling == SPEC_ROPE_BY_PARTS) {
            const double r = original_len * th / two_pi;
            const double g = std::min(1.0, std::max(0.0, (r - slow) / (fast - slow)));
            th *= (1.0 - g) / factor + g;
        }
        out_turns[i] = uint64_t(std::ldexp(th / two_pi, 64));  // th <= 1, so below 2^62
    }
    *out_scale = scaling == SPEC_ROPE_BY_PARTS ? float(0.1 * std::log(factor) + 1.0) : 1.f;
    return SPEC_OK;
}

spec_status spec_rope(const void* q, int q_heads, int64_t q_token_stride, int64_t q_head_stride,
                      void* out_q, int64_t oq_token_stride, int64_t oq_head_stride, const void* k,
                      int k_heads, int64_t k_token_stride, int64_t k_head_stride, void* out_k,
                      int64_t ok_token_stride, int64_t ok_head_stride, spec_dtype dtype, int D,
                      int64_t T, const int32_t* positions, const spec_rope_table* table,
                      int inverse, spec_stream_t stream) {
    if (T < 0 || q_heads < 0 || k_heads < 0 || q_heads > 65536 || k_heads > 65536 || D < 2 ||
        T > (1ll << 40) || !table)
        return SPEC_ERR_INVALID_ARG;
    if (dtype != SPEC_F32 && dtype != SPEC_BF16 && dtype != SPEC_F16) return SPEC_ERR_INVALID_ARG;
    if (D > 256 || D % 2) return SPEC_ERR_UNSUPPORTED;
    const spec_status ts = check_table(table, D);
    if (ts != SPEC_OK) return ts;
    if (T == 0 || q_heads + k_heads == 0) return SPEC_OK;
    if (!positions || (q_heads && (!q || !out_q)) || (k_heads && (!k || !out_k)))
        return SPEC_ERR_INVALID_ARG;
    const size_t es = dtype_bytes(dtype);
    if (!aligned(q, es) || !aligned(k, es) || !aligned(out_q, es) || !aligned(out_k, es) ||
        !aligned(positions, 4))
        return SPEC_ERR_UNSUPPORTED;
    RotArgs A = {};
    A.q = {q, out_q, q_token_stride, q_head_stride, oq_token_stride, oq_head_stride, q_heads};
    A.k = {k, out_k, k_token_stride, k_head_stride, ok_token_stride, ok_head_stride, k_heads};
    A.pos = positions;
    A.turns = reinterpret_cast<const unsigned long long*>(table->turns);
    A.half_rot = table->rot / 2;
    A.interleaved = table->layout == SPEC_ROPE_INTERLEAVED;
    A.scale = table->scale;
    A.sign = inverse ? -1.f : 1.f;
    A.D = D;
    A.T = T;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == SPEC_F32    ? launch_rotate_vec<float, false>(A, st)
                          : dtype == SPEC_BF16 ? launch_rotate_vec<__nv_bfloat16, false>(A, st)
                                               : launch_rotate_vec<__half, false>(A, st);
    return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

spec_status spec_kv_write(const spec_kv_cache* cache, const void* k, int64_t k_token_stride,
                          int64_t k_head_stride, const void* v, int64_t v_token_stride,
                          int64_t v_head_stride, spec_dtype dtype, int64_t T,
                          const int64_t* slots, const int32_t* positions,
                          const spec_rope_table* table, const void* q, int q_heads,
                          int64_t q_token_stride, int64_t q_head_stride, void* out_q,
                          int64_t oq_token_stride, int64_t oq_head_stride, int32_t* dev_status,
                          spec_stream_t stream) {
    const spec_status cs = check_cache(cache);
    if (cs != SPEC_OK) return cs;
    if (T < 0 || T > (1ll << 40) || q_heads < 0 || q_heads > 65536) return SPEC_ERR_INVALID_ARG;
    const bool e4 = cache->dtype == SPEC_E4M3;
    if (dtype != SPEC_F32 && dtype != SPEC_BF16 && dtype != SPEC_F16) return SPEC_ERR_INVALID_ARG;
    if (!e4 && int(dtype) != cache->dtype) return SPEC_ERR_INVALID_ARG;
    if (table) {
        const spec_status ts = check_table(table, cache->head_dim);
        if (ts != SPEC_OK) return ts;
        if (!positions && T > 0) return SPEC_ERR_INVALID_ARG;
    }
    if (q_heads && !table) return SPEC_ERR_INVALID_ARG;  // queries come along to be rotated
    if (T == 0) return SPEC_OK;
    if (!k || !v || !slots || (q_heads && (!q || !out_q))) return SPEC_ERR_INVALID_ARG;
    const size_t es = dtype_bytes(dtype);
    if (!aligned(k, es) || !aligned(v, es) || !aligned(q, es) || !aligned(out_q, es) ||
        !aligned(slots, 8) || !aligned(positions, 4) || !aligned(dev_status, 4))
        return SPEC_ERR_UNSUPPORTED;
    RotArgs A = {};
    if (q_heads)
        A.q = {q, out_q, q_token_stride, q_head_stride, oq_token_stride, oq_head_stride, q_heads};
    A.k = {k, nullptr, k_token_stride, k_head_stride, 0, 0, cache->heads};
    A.v = {v, nullptr, v_token_stride, v_head_stride, 0, 0, cache->heads};
    if (table) {
        A.pos = positions;
        A.turns = reinterpret_cast<const unsigned long long*>(table->turns);
        A.half_rot = table->rot / 2;
        A.interleaved = table->layout == SPEC_ROPE_INTERLEAVED;
        A.scale = table->scale;
    }
    A.sign = 1.f;
    A.D = cache->head_dim;
    A.T = T;
    A.c = view_of(*cache);
    A.slots = reinterpret_cast<const long long*>(slots);
    A.status = dev_status;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (e4)
        e = dtype == SPEC_F32    ? launch_rotate_vec<float, true>(A, st)
            : dtype == SPEC_BF16 ? launch_rotate_vec<__nv_bfloat16, true>(A, st)
                                 : launch_rotate_vec<__half, true>(A, st);
    else
        e = dtype == SPEC_BF16 ? launch_rotate_vec<__nv_bfloat16, false>(A, st)
                               : launch_rotate_vec<__half, false>(A, st);
    return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"

namespace {

template <typename C>
cudaError_t launch_read(const CacheView& c, int64_t T, const int64_t* slots, int dtype,
                        void* out_k, void* out_v, cudaStream_t st) {
    const long long n = T * c.heads * (c.D / 8);
    const unsigned grid = unsigned(std::min<long long>((n + 255) / 256, 1ll << 30));
    const long long* s = reinterpret_cast<const long long*>(slots);
    if (dtype == SPEC_F32)
        k_kv_read<C, float><<<grid, 256, 0, st>>>(c, T, s, static_cast<float*>(out_k),
                                                  static_cast<float*>(out_v));
    else if (dtype == SPEC_BF16)
        k_kv_read<C, __nv_bfloat16><<<grid, 256, 0, st>>>(
            c, T, s, static_cast<__nv_bfloat16*>(out_k), static_cast<__nv_bfloat16*>(out_v));
    else
        k_kv_read<C, __half><<<grid, 256, 0, st>>>(c, T, s, static_cast<__half*>(out_k),
                                                   static_cast<__half*>(out_v));
    return cudaGetLastError();
}

}  // namespace

extern "C" spec_status spec_kv_read(const spec_kv_cache* cache, int64_t T, const int64_t* slots,
                                    spec_dtype dtype, void* out_k, void* out_v,
                                    spec_stream_t stream) {
    const spec_status cs = check_cache(cache);
    if (cs != SPEC_OK) return cs;
    if (T < 0 || T > (1ll << 40)) return SPEC_ERR_INVALID_ARG;
    if (dtype != SPEC_F32 && dtype != SPEC_BF16 && dtype != SPEC_F16) return SPEC_ERR_INVALID_ARG;
    if (T == 0) return SPEC_OK;
    if (!slots || !out_k || !out_v) return SPEC_ERR_INVALID_ARG;
    if (!aligned(slots, 8) || !aligned(out_k, 16) || !aligned(out_v, 16))
        return SPEC_ERR_UNSUPPORTED;
    const CacheView c = view_of(*cache);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e =
        cache->dtype == SPEC_E4M3
            ? launch_read<uint8_t>(c, T, slots, dtype, out_k, out_v, st)
        : cache->dtype == SPEC_BF16
            ? launch_read<__nv_bfloat16>(c, T, slots, dtype, out_k, out_v, st)
            : launch_read<__half>(c, T, slots, dtype, out_k, out_v, st);
    return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
