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
// The kernels are bound by memory: every byte is read and written once.  32771 tokens
// of 40 heads of 128 channels, half of them turned, take 99 us (1.00 of the measured
// copy rate), all of them turned in half layout 103 (0.96); 4608 tokens of 48 heads, keys
// and values to 8 bits, 21 (0.7); reading these back 8.  80 registers a thread (three CTAs an
// SM) are not enough for pairs half a head apart in vectors of 8, nor for e4m3 rows in
// vectors of 16: they spill 48 to 112 bytes a thread.
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
// token; E4: the cache is e4m3 (else of type T); PAIR: half layout (else
// interleaved, or nothing turns).
template <typename T, int VEC, int IP, bool E4, bool PAIR>
__global__ void __launch_bounds__(ROT_THREADS, 3) k_rotate(const __grid_constant__ RotArgs A) {
    begin_after_previous();
    const int lane = threadIdx.x % IP;
    const long long t = blockIdx.x * (long long)(ROT_THREADS / IP) + threadIdx.x / IP;
    if (t >= A.T) return;
    const unsigned gmask = IP == 32 ? 0xffffffffu : ((1u << IP) - 1u) << (((threadIdx.x & 31) / IP) * IP);
    const int hr = A.half_rot, h0 = blockIdx.y * A.share, h1 = h0 + A.share;
    // this lane's item of a head that turns, and of one that does not
    Place pt = {lane * VEC, 0, lane * VEC < A.D, false}, pp = pt;
    if (PAIR && (lane + IP) * VEC < A.D) pp.second = IP * VEC;
    if (!PAIR) {
        pt.turns = pt.off < 2 * hr;
    } else {
        const int r = hr / VEC;
        pt.turns = lane < r;
        if (pt.turns) pt.second = hr;
        else pt.off = 2 * hr + (lane - r) * VEC;
        pt.on = pt.off < A.D;
    }
    // UH heads' items from `in`, as many as there are
    constexpr int UH = 128 / (VEC * int(sizeof(T)) * (PAIR ? 2 : 1));
    Words<T, VEC> x[UH], y[PAIR ? UH : 1];
    auto load = [&](const T* in, long long ih, const Place& p, int n) {
#pragma unroll
        for (int u = 0; u < UH; ++u)
            if (p.on && u < n) {
                x[u] = *reinterpret_cast<const Words<T, VEC>*>(in + u * ih);
                if (PAIR && p.second) y[u] = *reinterpret_cast<const Words<T, VEC>*>(in + u * ih + p.second);
            }
    };
    // The share's heads of each tensor, and where they go.  Nothing turns, or pairs lie
    // side by side: one flat loop, whose first loads are under way while the slot is
    // read and the angles are made (20011 tokens' keys and values to 8 bits and back 57
    // -> 50 us).  Pairs half a head apart: nested loops that load as they go, since
    // angles and two vectors an item together would spill still more (11128 tokens of
    // narrow heads 52 us, by the flat loop 65).
    auto tensor = [&](int kind) -> const Heads& { return kind == 0 ? A.q : kind == 1 ? A.k : A.v; };
    int kind = 0, h = 0, hi = 0;
    auto first_of = [&]() {  // of `kind` or the next that has some
        for (; kind < 3; ++kind) {
            const int base = kind == 0 ? 0 : kind == 1 ? A.q.n : A.q.n + A.k.n;
            h = max(h0 - base, 0);
            hi = min(h1 - base, tensor(kind).n);
            if (h < hi) break;
        }
    };
    auto load_here = [&]() {
        const Heads& X = tensor(kind);
        const Place& p = kind != 2 && hr ? pt : pp;
        load(static_cast<const T*>(X.in) + t * X.it + h * X.ih + p.off, X.ih, p, hi - h);
    };
    if constexpr (!PAIR) {
        first_of();
        load_here();
    }
    const SlotRow sr = slot_row(A, t, lane == 0 && blockIdx.y == 0);
    constexpr int NT = PAIR ? VEC : VEC / 2;  // angles of an item, at most
    float cs[NT], sn[NT];
    if (hr && pt.turns) {
        const int pos = __ldg(A.pos + t);
#pragma unroll
        for (int e = 0; e < NT; ++e) {
            angle(__ldg(A.turns + lane * NT + e), pos, cs[e], sn[e]);
            cs[e] *= A.scale;
            sn[e] *= A.scale * A.sign;
        }
    }

    // UH heads from h on: to `out`, or (bytes, scales) as e4m3
    auto put = [&](int h, int hi, const Place& p, T* out, long long oh, uint8_t* bytes, uint8_t* scales) {
#pragma unroll
        for (int u = 0; u < UH; ++u) {
            if (h + u >= hi) break;  // the same for the whole group
            float va[VEC], vb[PAIR ? VEC : 1];
#pragma unroll
            for (int e = 0; e < VEC / 2; ++e) {
                const float2 a = get2(x[u], e);
                va[2 * e] = a.x;
                va[2 * e + 1] = a.y;
                if (PAIR) {
                    const float2 b = get2(y[PAIR ? u : 0], e);
                    vb[PAIR ? 2 * e : 0] = b.x;
                    vb[PAIR ? 2 * e + 1 : 0] = b.y;
                }
            }
            if (p.turns) {
                if constexpr (PAIR) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float a = va[e], b = vb[e];
                        va[e] = a * cs[e] - b * sn[e];
                        vb[e] = a * sn[e] + b * cs[e];
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < VEC / 2; ++e) {
                        const float a = va[2 * e], b = va[2 * e + 1];
                        va[2 * e] = a * cs[e] - b * sn[e];
                        va[2 * e + 1] = a * sn[e] + b * cs[e];
                    }
                }
            }
            if (E4 && bytes) {
                // (a maximum drops NaN, which converts to NaN; an infinity shows in it)
                auto widest = [&](auto&& size) {
                    float m = 0.f;
                    if (p.on) {
#pragma unroll
                        for (int e = 0; e < VEC; ++e) m = fmaxf(m, size(va[e]));
                        if (PAIR && p.second) {
#pragma unroll
                            for (int e = 0; e < VEC; ++e) m = fmaxf(m, size(vb[PAIR ? e : 0]));
                        }
                    }
#pragma unroll
                    for (int o = IP / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(gmask, m, o, IP));
                    return m;
                };
                float m = widest([](float f) { return fabsf(f); });
                const bool odd = m == INFINITY;  // seldom: then finite values alone count
                if (odd) m = widest([](float f) { return finite_abs(f); });
                const int ex = e4m3_exponent(m);
                const float down = exp2_int(-ex);
                if (p.on) {
                    Words<uint8_t, VEC> a, b;
                    auto pack = [&](auto&& two) {
#pragma unroll
                        for (int e = 0; e < VEC / 4; ++e) {
                            a.w[e] = two(va[4 * e] * down, va[4 * e + 1] * down) |
                                     uint32_t(two(va[4 * e + 2] * down, va[4 * e + 3] * down)) << 16;
                            if constexpr (PAIR)
                                b.w[e] = two(vb[4 * e] * down, vb[4 * e + 1] * down) |
                                         uint32_t(two(vb[4 * e + 2] * down, vb[4 * e + 3] * down)) << 16;
                            else b.w[e] = 0;
                        }
                    };
                    if (__builtin_expect(odd, 0)) {
                        pack([](float lo, float hi) { return pack_e4m3x2(lo, hi); });
                    } else {
                        pack([](float lo, float hi) {
                            uint16_t r;
                            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
                            return r;
                        });
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
                    set2(a, e, va[2 * e], va[2 * e + 1]);
                    if constexpr (PAIR) set2(b, e, vb[2 * e], vb[2 * e + 1]);
                    else set2(b, e, 0.f, 0.f);
                }
                T* at = out + (h + u) * oh + p.off;
                *reinterpret_cast<Words<T, VEC>*>(at) = a;
                if (PAIR && p.second) *reinterpret_cast<Words<T, VEC>*>(at + p.second) = b;
            }
        }
    };
    // the tensor `kind`: f(its heads, an item's place, where they go)
    auto with = [&](int kind, auto&& f) {
        const bool cached = A.slots && kind;
        if (cached && sr.row < 0) return;
        const Heads& X = tensor(kind);
        const Place p = kind != 2 && hr ? pt : pp;
        T* out = cached ? static_cast<T*>(kind == 1 ? A.c.k : A.c.v) + (E4 ? 0 : sr.row)
                        : static_cast<T*>(X.out) + t * X.ot;
        uint8_t* bytes = E4 && cached ? static_cast<uint8_t*>(kind == 1 ? A.c.k : A.c.v) + sr.row : nullptr;
        f(X, p, out, cached ? A.c.head_stride : X.oh, bytes,
          E4 && cached ? (kind == 1 ? A.c.ks : A.c.vs) + sr.scale : nullptr);
    };
    if constexpr (PAIR) {
#pragma unroll 1
        for (int k = 0; k < 3; ++k) {
            const int base = k == 0 ? 0 : k == 1 ? A.q.n : A.q.n + A.k.n;
            const int lo = max(h0 - base, 0), end = min(h1 - base, tensor(k).n);
            if (lo >= end) continue;
            with(k, [&](const Heads& X, const Place& p, T* out, long long oh, uint8_t* bytes, uint8_t* scales) {
                const T* in = static_cast<const T*>(X.in) + t * X.it + lo * X.ih + p.off;
#pragma unroll 1
                for (int i = lo; i < end; i += UH) {
                    load(in, X.ih, p, end - i);
                    in += UH * X.ih;
                    put(i, end, p, out, oh, bytes, scales);
                }
            });
        }
    } else {
#pragma unroll 1
        while (kind < 3) {
            with(kind, [&](const Heads&, const Place& p, T* out, long long oh, uint8_t* bytes, uint8_t* scales) {
                put(h, hi, p, out, oh, bytes, scales);
            });
            h += UH;
            if (h >= hi) {
                ++kind;
                first_of();
            }
            if (kind < 3) load_here();
        }
    }
}

// Any strides, alignment and even rot: a warp a (token, head), a lane one pair
// or one value that does not turn at a time; an e4m3 row is read twice.
template <typename T, bool E4>
__global__ void __launch_bounds__(ROT_THREADS) k_rotate_any(const __grid_constant__ RotArgs A) {
    begin_after_previous();
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

// Rows of T slots: one thread per 16 bytes of a (token, head)'s row as it is
// written, so that a warp's stores leave no gaps.  I: the type
// of the indexes (32 bits where they are enough: a division of 64 costs more than
// the copy).
template <typename C, typename T, typename I>
__global__ void __launch_bounds__(256) k_kv_read(const __grid_constant__ CacheView c, long long T_,
                                                 const long long* slots, T* out_k, T* out_v) {
    begin_after_previous();
    constexpr int VEC = 16 / sizeof(T);
    const I vecs = c.D / VEC, heads = c.heads, n = I(T_) * heads * vecs;
    for (I i = blockIdx.x * I(256) + threadIdx.x; i < n; i += gridDim.x * I(256)) {
        const I th = i / vecs, t = th / heads;
        const int d = int(i - th * vecs) * VEC, h = int(th - t * heads);
        const long long slot = slots[t];
        Words<C, VEC> k, v;
        float fk = 1.f, fv = 1.f;
#pragma unroll
        for (int e = 0; e < VEC * int(sizeof(C)) / 4; ++e) k.w[e] = v.w[e] = 0;
        if (slot >= 0 && slot < c.slots) {
            const long long p = sizeof(I) == 4 ? (long long)(uint32_t(slot) / uint32_t(c.page)) : slot / c.page;
            const int o = int(slot - p * c.page);
            const long long at = p * c.page_stride + h * c.head_stride + o * c.token_stride + d;
            k = *reinterpret_cast<const Words<C, VEC>*>(static_cast<const C*>(c.k) + at);
            v = *reinterpret_cast<const Words<C, VEC>*>(static_cast<const C*>(c.v) + at);
            if constexpr (sizeof(C) == 1) {
                const long long sr = (p * c.heads + h) * c.page + o;
                fk = exp2_int(min(max(int(c.ks[sr]), 1), 253) - 127);
                fv = exp2_int(min(max(int(c.vs[sr]), 1), 253) - 127);
            }
        }
        auto write = [&](const Words<C, VEC>& x, float f, T* out) {
            Words<T, VEC> w;
#pragma unroll
            for (int e = 0; e < VEC / 2; ++e) {
                float2 a;
                if constexpr (sizeof(C) == 1) {
                    const uint32_t b = e4m3x2_to_f16x2(uint16_t(x.w[e / 2] >> (16 * (e & 1))));
                    a = __half22float2(*reinterpret_cast<const __half2*>(&b));
                    a.x *= f;
                    a.y *= f;
                } else {
                    a = get2(x, e);
                }
                set2(w, e, a.x, a.y);
            }
            *reinterpret_cast<Words<T, VEC>*>(out + (long long)i * VEC) = w;
        };
        write(k, fk, out_k);
        write(v, fv, out_v);
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
    // once, where that leaves every SM 3072 lanes (four times what it holds); with
    // fewer tokens a share of the heads, twice as many as have their loads in flight
    // together (UH) while that leaves every SM 768 lanes, else UH, as where nothing
    // turns, and single heads where even that leaves SMs without work.
    constexpr int UH = 128 / (VEC * int(sizeof(T)) * (PAIR ? 2 : 1));
    const long long lanes = A.T * ip;
    int share = A.half_rot ? (H + UH - 1) / UH * UH : UH;
    while (share > 2 * UH && lanes * ((H + share - 1) / share) < 3072ll * sms) share -= UH;
    while (share > UH && lanes * ((H + share - 1) / share) < 768ll * sms) share -= UH;
    if (share == UH && lanes * ((H + UH - 1) / UH) < 256ll * sms) share = 1;
    A.share = std::max(share, (H + 65534) / 65535);  // blockIdx.y ends at 65534
    const long long gx = (A.T + ROT_THREADS / ip - 1) / (ROT_THREADS / ip);
    if (gx > 0x7fffffffll) return cudaErrorInvalidValue;
    const dim3 grid(unsigned(gx), unsigned((H + A.share - 1) / A.share));
    auto* kernel = ip == 4    ? k_rotate<T, VEC, 4, E4, PAIR>
                   : ip == 8  ? k_rotate<T, VEC, 8, E4, PAIR>
                   : ip == 16 ? k_rotate<T, VEC, 16, E4, PAIR>
                              : k_rotate<T, VEC, 32, E4, PAIR>;
    return launch_behind(kernel, grid, ROT_THREADS, 0, st, A);
}

template <typename T, bool E4>
cudaError_t launch_rotate_vec(const RotArgs& A, cudaStream_t st) {
    // vectors of 16 elements, 8 or 4, where every offset of the call is a
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
    if constexpr (E4 && sizeof(T) == 2)  // bytes then go out 16 at a time too
        if (!pair && ok(16)) return launch_rotate<T, 16, E4, false>(A, st);
    if (ok(8)) return pair ? launch_rotate<T, 8, E4, true>(A, st) : launch_rotate<T, 8, E4, false>(A, st);
    if (ok(4)) return pair ? launch_rotate<T, 4, E4, true>(A, st) : launch_rotate<T, 4, E4, false>(A, st);
    const long long warps = A.T * (A.q.n + A.k.n + A.v.n), grid = (warps + ROT_THREADS / 32 - 1) / (ROT_THREADS / 32);
    if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
    return launch_behind(k_rotate_any<T, E4>, dim3(unsigned(grid)), ROT_THREADS, 0, st, A);
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
    const long long n = T_ * c.heads * (c.D / (16 / int(sizeof(T))));
    const unsigned grid = unsigned(std::min<long long>((n + 255) / 256, 1ll << 22));
    const long long* s = reinterpret_cast<const long long*>(slots);
    T *k = static_cast<T*>(out_k), *v = static_cast<T*>(out_v);
    auto* kernel = n < (1ll << 31) && c.slots < (1ll << 32) ? k_kv_read<C, T, uint32_t> : k_kv_read<C, T, long long>;
    return launch_behind(kernel, dim3(grid), 256, 0, st, c, (long long)T_, s, k, v);
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
