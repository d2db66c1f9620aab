// rope.cu -- rotary positions, and the cache rows written and read.
//
// The heads of a token are turned by its position's angles and stored: to a
// tensor (spec_rope), or to the token's cache slot, as they are or in 8 bits
// (spec_kv_write).
//
// k_rotate (aligned tensors): IP lanes take a token and a share of its heads, a
// lane one item of every head:
//   of the rotated part VEC pairs (half layout: two vectors rot / 2 channels
//     apart; interleaved: one vector of VEC / 2 pairs), of the rest one vector;
//   of a head that does not turn up to two vectors.
// So a lane computes its sines and cosines once for all heads and keeps them in
// registers, its addresses advance by a stride, the loads of several heads are in
// flight together (128 bytes a lane: HBM's latency at its rate is some 50 KB an
// SM), and an e4m3 row's maximum is a shuffle within the IP lanes.
// k_rotate_any takes every other alignment, one value at a time.
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
#include <type_traits>

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
    int share;  // heads a group of lanes takes (blockIdx.y: which)
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

// Where an item's vectors lie in a head: at `off`, and `second` channels on
// (0: one vector).
struct Place {
    int off, second;
    bool on, turns;
};

// A token's row in the cache (element offset of head 0, or -1: not written) and
// its scales' place.
struct SlotRow {
    long long row, scale;
};
__device__ __forceinline__ SlotRow slot_row(const RotArgs& A, long long t, bool report) {
    SlotRow r = {-1, 0};
    if (!A.slots) return r;
    const long long slot = A.slots[t];
    if (slot >= A.c.slots && report && A.status) atomicOr(A.status, int(SPEC_BADBIT_PAGE));
    if (slot >= 0 && slot < A.c.slots) {
        const long long p = A.c.slots <= 0x7fffffff ? (long long)(uint32_t(slot) / uint32_t(A.c.page)) : slot / A.c.page;
        const int o = int(slot - p * A.c.page);
        r.row = p * A.c.page_stride + o * A.c.token_stride;
        r.scale = p * A.c.heads * A.c.page + o;
    }
    return r;
}

// VEC elements as 32-bit words (a vector of 16-bit elements would take a register
// an element).
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC < 16 ? sizeof(T) * VEC : 16) Words {
    uint32_t w[VEC * sizeof(T) / 4];
};
// elements 2 e and 2 e + 1
template <typename T, int VEC>
__device__ __forceinline__ float2 get2(const Words<T, VEC>& x, int e) {
    if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(x.w[2 * e]), __uint_as_float(x.w[2 * e + 1]));
    else if constexpr (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<const __half2*>(&x.w[e]));
    else return make_float2(bf16_lo(x.w[e]), bf16_hi(x.w[e]));
}
template <typename T, int VEC>
__device__ __forceinline__ void set2(Words<T, VEC>& x, int e, float a, float b) {
    if constexpr (sizeof(T) == 4) {
        x.w[2 * e] = __float_as_uint(a);
        x.w[2 * e + 1] = __float_as_uint(b);
    } else if constexpr (std::is_same<T, __half>::value) {
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(x.w[e]) : "f"(b), "f"(a));
    } else {
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(x.w[e]) : "f"(b), "f"(a));
    }
}

// T: element type of the tensors; VEC: elements of a vector; IP: lanes of a
// token; E4: the cache is e4m3 (else of type T); PAIR: some item has two vectors.
template <typename T, int VEC, int IP, bool E4, bool PAIR>
__global__ void __launch_bounds__(ROT_THREADS, 3) k_rotate(const __grid_constant__ RotArgs A) {
    const int lane = threadIdx.x % IP;
    const long long t = blockIdx.x * (long long)(ROT_THREADS / IP) + threadIdx.x / IP;
    if (t >= A.T) return;
    const unsigned gmask = IP == 32 ? 0xffffffffu : ((1u << IP) - 1u) << (((threadIdx.x & 31) / IP) * IP);
    const int hr = A.half_rot, h0 = blockIdx.y * A.share, h1 = h0 + A.share;
    const SlotRow sr = slot_row(A, t, lane == 0 && blockIdx.y == 0);

    // this lane's item of a head that turns, and of one that does not
    Place pt = {lane * VEC, 0, lane * VEC < A.D, false}, pp = pt;
    if (PAIR && (lane + IP) * VEC < A.D) pp.second = IP * VEC;
    if (A.interleaved) {
        pt.turns = pt.off < 2 * hr;
    } else {
        const int r = hr / VEC;
        pt.turns = lane < r;
        if (pt.turns) pt.second = hr;
        else pt.off = 2 * hr + (lane - r) * VEC;
        pt.on = pt.off < A.D;
    }
    constexpr int NT = PAIR ? VEC : VEC / 2;  // angles of an item, at most
    float cs[NT], sn[NT];
    if (hr && pt.turns) {
        const int pos = __ldg(A.pos + t);
        const int n = A.interleaved ? VEC / 2 : VEC;
#pragma unroll
        for (int e = 0; e < NT; ++e)
            if (e < n) {
                angle(__ldg(A.turns + lane * n + e), pos, cs[e], sn[e]);
                cs[e] *= A.scale;
                sn[e] *= A.scale * A.sign;
            }
    }

    // heads [lo, hi) of one tensor: to `out`, or (bytes, scales) as e4m3
    auto heads = [&](const Heads& X, int lo, int hi, const Place& p, T* out, long long oh, uint8_t* bytes,
                     uint8_t* scales) {
        const T* in = static_cast<const T*>(X.in) + t * X.it + lo * X.ih + p.off;
        constexpr int UH = 128 / (VEC * int(sizeof(T)) * (PAIR ? 2 : 1));
#pragma unroll 1
        for (int h = lo; h < hi; h += UH) {
            Words<T, VEC> x[UH], y[PAIR ? UH : 1];
#pragma unroll
            for (int u = 0; u < UH; ++u)
                if (p.on && h + u < hi) {
                    x[u] = *reinterpret_cast<const Words<T, VEC>*>(in + u * X.ih);
                    if (PAIR && p.second) y[u] = *reinterpret_cast<const Words<T, VEC>*>(in + u * X.ih + p.second);
                }
            in += UH * X.ih;
#pragma unroll
            for (int u = 0; u < UH; ++u) {
                if (h + u >= hi) break;  // the same for the whole group
                // elements 2 e and 2 e + 1 of the first vector and of the second
                auto four = [&](int e, float (&f)[4]) {
                    const float2 a2 = get2(x[u], e), b2 = PAIR ? get2(y[PAIR ? u : 0], e) : make_float2(0.f, 0.f);
                    f[0] = a2.x;
                    f[1] = a2.y;
                    f[2] = b2.x;
                    f[3] = b2.y;
                    if (!p.turns) return;
                    if (A.interleaved) {
                        const float a = f[0], b = f[1];
                        f[0] = a * cs[e] - b * sn[e];
                        f[1] = a * sn[e] + b * cs[e];
                    } else if (PAIR) {
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const int i = PAIR ? 2 * e + z : 0;
                            const float a = f[z], b = f[2 + z];
                            f[z] = a * cs[i] - b * sn[i];
                            f[2 + z] = a * sn[i] + b * cs[i];
                        }
                    }
                };
                float f[4];
                if (E4 && bytes) {
                    float m = 0.f;
                    if (p.on) {
#pragma unroll
                        for (int e = 0; e < VEC / 2; ++e) {
                            four(e, f);
                            m = fmaxf(m, fmaxf(finite_abs(f[0]), finite_abs(f[1])));
                            if (PAIR && p.second) m = fmaxf(m, fmaxf(finite_abs(f[2]), finite_abs(f[3])));
                        }
                    }
#pragma unroll
                    for (int o = IP / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(gmask, m, o, IP));
                    const int ex = e4m3_exponent(m);
                    if (p.on) {
                        Words<uint8_t, VEC> a, b;
#pragma unroll
                        for (int e = 0; e < VEC / 4; ++e) {
                            float g[4];
                            four(2 * e, f);
                            four(2 * e + 1, g);
                            a.w[e] = pack_e4m3x2(e4m3_scaled(f[0], ex), e4m3_scaled(f[1], ex)) |
                                     uint32_t(pack_e4m3x2(e4m3_scaled(g[0], ex), e4m3_scaled(g[1], ex))) << 16;
                            if (PAIR)
                                b.w[e] = pack_e4m3x2(e4m3_scaled(f[2], ex), e4m3_scaled(f[3], ex)) |
                                         uint32_t(pack_e4m3x2(e4m3_scaled(g[2], ex), e4m3_scaled(g[3], ex))) << 16;
                        }
                        uint8_t* at = bytes + (h + u) * A.c.head_stride + p.off;
                        *reinterpret_cast<Words<uint8_t, VEC>*>(at) = a;
                        if (PAIR && p.second) *reinterpret_cast<Words<uint8_t, VEC>*>(at + p.second) = b;
                    }
                    if (lane == 0) scales[(long long)(h + u) * A.c.page] = uint8_t(ex + 127);
                } else if (p.on) {
                    Words<T, VEC> a, b;
#pragma unroll
                    for (int e = 0; e < VEC / 2; ++e) {
                        four(e, f);
                        set2(a, e, f[0], f[1]);
                        if (PAIR) set2(b, e, f[2], f[3]);
                    }
                    T* at = out + (h + u) * oh + p.off;
                    *reinterpret_cast<Words<T, VEC>*>(at) = a;
                    if (PAIR && p.second) *reinterpret_cast<Words<T, VEC>*>(at + p.second) = b;
                }
            }
        }
    };
    // one loop over the three tensors, so that its code is there once
#pragma unroll 1
    for (int kind = 0; kind < 3; ++kind) {
        const Heads& X = kind == 0 ? A.q : kind == 1 ? A.k : A.v;
        const int base = kind == 0 ? 0 : kind == 1 ? A.q.n : A.q.n + A.k.n;
        const int lo = max(h0 - base, 0), hi = min(h1 - base, X.n);
        const bool cached = A.slots && kind;
        if (lo >= hi || (cached && sr.row < 0)) continue;
        const bool turning = kind != 2 && hr;
        const Place p = turning ? pt : pp;
        T* out = cached ? static_cast<T*>(kind == 1 ? A.c.k : A.c.v) + (E4 ? 0 : sr.row)
                        : static_cast<T*>(X.out) + t * X.ot;
        uint8_t* bytes = E4 && cached ? static_cast<uint8_t*>(kind == 1 ? A.c.k : A.c.v) + sr.row : nullptr;
        heads(X, lo, hi, p, out, cached ? A.c.head_stride : X.oh, bytes,
              E4 && cached ? (kind == 1 ? A.c.ks : A.c.vs) + sr.scale : nullptr);
    }
}

// Any strides, alignment and even rot: a warp a (token, head), a lane one pair
// or one value that does not turn at a time; an e4m3 row is read twice.
template <typename T, bool E4>
__global__ void __launch_bounds__(ROT_THREADS) k_rotate_any(const __grid_constant__ RotArgs A) {
    const int lane = threadIdx.x & 31, H = A.q.n + A.k.n + A.v.n, hr = A.half_rot;
    const long long w = blockIdx.x * (long long)(ROT_THREADS / 32) + (threadIdx.x >> 5);
    if (w >= A.T * H) return;
    const long long t = w / H;
    const int h = int(w - t * H), kind = h < A.q.n ? 0 : h < A.q.n + A.k.n ? 1 : 2;
    const int hh = kind == 0 ? h : kind == 1 ? h - A.q.n : h - A.q.n - A.k.n;
    const SlotRow sr = slot_row(A, t, lane == 0 && h == 0);
    const bool cached = A.slots && kind, turning = kind != 2 && hr;
    if (cached && sr.row < 0) return;
    const Heads& X = kind == 0 ? A.q : kind == 1 ? A.k : A.v;
    const T* in = static_cast<const T*>(X.in) + t * X.it + hh * X.ih;
    const int pairs = turning ? hr : 0, rest = A.D - 2 * pairs;
    const int pos = turning ? A.pos[t] : 0;
    // item i: a pair's two values and channels, or one of the rest (second -1)
    auto get = [&](int i, int& a, int& b, float& x, float& y) {
        if (i < pairs) {
            a = A.interleaved ? 2 * i : i;
            b = A.interleaved ? a + 1 : i + hr;
            float c, s;
            angle(A.turns[i], pos, c, s);
            c *= A.scale;
            s *= A.scale * A.sign;
            const float u = to_f32(in[a]), v = to_f32(in[b]);
            x = u * c - v * s;
            y = u * s + v * c;
        } else {
            a = i + pairs;
            b = -1;
            x = to_f32(in[a]);
            y = 0.f;
        }
    };
    int a, b, ex = 0;
    float x, y;
    if (E4 && cached) {
        float m = 0.f;
        for (int i = lane; i < pairs + rest; i += 32) {
            get(i, a, b, x, y);
            m = fmaxf(m, fmaxf(finite_abs(x), finite_abs(y)));
        }
        ex = e4m3_exponent(warp_max(m));
        if (lane == 0) ((kind == 1 ? A.c.ks : A.c.vs) + sr.scale)[(long long)hh * A.c.page] = uint8_t(ex + 127);
    }
    for (int i = lane; i < pairs + rest; i += 32) {
        get(i, a, b, x, y);
        if (E4 && cached) {
            uint8_t* out = static_cast<uint8_t*>(kind == 1 ? A.c.k : A.c.v) + sr.row + hh * A.c.head_stride;
            const uint16_t o = pack_e4m3x2(e4m3_scaled(x, ex), e4m3_scaled(y, ex));
            out[a] = uint8_t(o);
            if (b >= 0) out[b] = uint8_t(o >> 8);
        } else {
            T* out = cached ? static_cast<T*>(kind == 1 ? A.c.k : A.c.v) + sr.row + hh * A.c.head_stride
                            : static_cast<T*>(X.out) + t * X.ot + hh * X.oh;
            out[a] = from_f32<T>(x);
            if (b >= 0) out[b] = from_f32<T>(y);
        }
    }
}

// Rows of T slots: one thread per 8 channels of a (token, head).  I: the type
// of the indexes (32 bits where they are enough: a division of 64 costs more than
// the copy).
template <typename C, typename T, typename I>
__global__ void __launch_bounds__(256) k_kv_read(const __grid_constant__ CacheView c, long long T_,
                                                 const long long* slots, T* out_k, T* out_v) {
    const I vecs = c.D / 8, heads = c.heads, n = I(T_) * heads * vecs;
    for (I i = blockIdx.x * I(256) + threadIdx.x; i < n; i += gridDim.x * I(256)) {
        const I th = i / vecs, t = th / heads;
        const int d = int(i - th * vecs) * 8, h = int(th - t * heads);
        const long long slot = slots[t];
        Vec<T, 8> ok, ov;
#pragma unroll
        for (int e = 0; e < 8; ++e) ok.e[e] = ov.e[e] = from_f32<T>(0.f);
        if (slot >= 0 && slot < c.slots) {
            const long long p = sizeof(I) == 4 ? (long long)(uint32_t(slot) / uint32_t(c.page)) : slot / c.page;
            const int o = int(slot - p * c.page);
            const long long at = p * c.page_stride + h * c.head_stride + o * c.token_stride + d;
            if constexpr (sizeof(C) == 1) {
                const long long sr = (p * c.heads + h) * c.page + o;
                const float fk = exp2_int(min(max(int(c.ks[sr]), 1), 253) - 127),
                            fv = exp2_int(min(max(int(c.vs[sr]), 1), 253) - 127);
                const Vec<uint16_t, 4> k = load_vec<uint16_t, 4>(
                    reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(c.k) + at));
                const Vec<uint16_t, 4> v = load_vec<uint16_t, 4>(
                    reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(c.v) + at));
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t wk = e4m3x2_to_f16x2(k.e[e]), wv = e4m3x2_to_f16x2(v.e[e]);
                    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&wk));
                    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&wv));
                    ok.e[2 * e] = from_f32<T>(a.x * fk);
                    ok.e[2 * e + 1] = from_f32<T>(a.y * fk);
                    ov.e[2 * e] = from_f32<T>(b.x * fv);
                    ov.e[2 * e + 1] = from_f32<T>(b.y * fv);
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
        store_vec<T, 8>(out_k + (long long)i * 8, ok);
        store_vec<T, 8>(out_v + (long long)i * 8, ov);
    }
}

// Lanes that a token's heads need at VEC elements a vector (more than 32: none);
// two vectors an item only where pairs are half a head apart.
int lanes_for(const RotArgs& A, int vec) {
    if (!A.half_rot || A.interleaved) return A.D / vec;
    return std::max(A.half_rot / vec + (A.D - 2 * A.half_rot) / vec, A.v.n ? (A.D / vec + 1) / 2 : 0);
}

template <typename T, int VEC, bool E4, bool PAIR>
cudaError_t launch_rotate(RotArgs A, cudaStream_t st) {
    const int want = lanes_for(A, VEC), ip = want <= 4 ? 4 : want <= 8 ? 8 : want <= 16 ? 16 : 32;
    const int H = A.q.n + A.k.n + A.v.n, sms = sm_count();
    if (sms <= 0) return cudaErrorUnknown;
    // A group takes all heads of its token, so that sines and cosines are computed
    // once, where that leaves every SM 1536 lanes; with fewer tokens a share of the
    // heads, four at least (whose loads are in flight together), and single heads
    // where even that leaves SMs without work.
    int shares = 1;
    const long long lanes = A.T * ip;
    while (shares * 4 < H && lanes * shares < 1536ll * sms) ++shares;
    if (shares * 4 >= H && lanes * shares < 256ll * sms) shares = H;
    A.share = (H + shares - 1) / shares;
    const long long gx = (A.T + ROT_THREADS / ip - 1) / (ROT_THREADS / ip);
    if (gx > 0x7fffffffll || (H + A.share - 1) / A.share > 65535) return cudaErrorInvalidValue;
    const dim3 grid(unsigned(gx), unsigned((H + A.share - 1) / A.share));
    if (ip == 4) k_rotate<T, VEC, 4, E4, PAIR><<<grid, ROT_THREADS, 0, st>>>(A);
    else if (ip == 8) k_rotate<T, VEC, 8, E4, PAIR><<<grid, ROT_THREADS, 0, st>>>(A);
    else if (ip == 16) k_rotate<T, VEC, 16, E4, PAIR><<<grid, ROT_THREADS, 0, st>>>(A);
    else k_rotate<T, VEC, 32, E4, PAIR><<<grid, ROT_THREADS, 0, st>>>(A);
    return cudaGetLastError();
}

template <typename T, bool E4>
cudaError_t launch_rotate_vec(const RotArgs& A, cudaStream_t st) {
    // vectors of 8 elements or of 4, where every offset of the call is a
    // multiple of that; else one value at a time
    auto ok = [&](int vec) {
        const size_t a = std::min<size_t>(16, vec * sizeof(T));
        auto side = [&](const Heads& h, bool out) {
            if (!h.n) return true;
            if (!aligned(h.in, a) || h.it % vec || h.ih % vec) return false;
            return !out || (aligned(h.out, a) && h.ot % vec == 0 && h.oh % vec == 0);
        };
        if (A.D % vec || (A.interleaved ? 2 * A.half_rot : A.half_rot) % vec || lanes_for(A, vec) > 32) return false;
        return side(A.q, true) && side(A.k, !A.slots) && side(A.v, false);
    };
    const bool pair = A.half_rot && !A.interleaved;
    if (ok(8)) return pair ? launch_rotate<T, 8, E4, true>(A, st) : launch_rotate<T, 8, E4, false>(A, st);
    if (ok(4)) return pair ? launch_rotate<T, 4, E4, true>(A, st) : launch_rotate<T, 4, E4, false>(A, st);
    const long long warps = A.T * (A.q.n + A.k.n + A.v.n), grid = (warps + ROT_THREADS / 32 - 1) / (ROT_THREADS / 32);
    if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
    k_rotate_any<T, E4><<<unsigned(grid), ROT_THREADS, 0, st>>>(A);
    return cudaGetLastError();
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

template <typename C, typename T>
cudaError_t launch_read_to(const CacheView& c, int64_t T_, const int64_t* slots, void* out_k, void* out_v,
                           cudaStream_t st) {
    const long long n = T_ * c.heads * (c.D / 8);
    const unsigned grid = unsigned(std::min<long long>((n + 255) / 256, 1ll << 22));
    const long long* s = reinterpret_cast<const long long*>(slots);
    T *k = static_cast<T*>(out_k), *v = static_cast<T*>(out_v);
    if (n < (1ll << 31) && c.slots < (1ll << 32)) k_kv_read<C, T, uint32_t><<<grid, 256, 0, st>>>(c, T_, s, k, v);
    else k_kv_read<C, T, long long><<<grid, 256, 0, st>>>(c, T_, s, k, v);
    return cudaGetLastError();
}
template <typename C>
cudaError_t launch_read(const CacheView& c, int64_t T, const int64_t* slots, int dtype,
                        void* out_k, void* out_v, cudaStream_t st) {
    if (dtype == SPEC_F32) return launch_read_to<C, float>(c, T, slots, out_k, out_v, st);
    if (dtype == SPEC_BF16) return launch_read_to<C, __nv_bfloat16>(c, T, slots, out_k, out_v, st);
    return launch_read_to<C, __half>(c, T, slots, out_k, out_v, st);
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
