// rotate.cuh -- k_rotate and k_rotate_any: the heads of tokens turned by their positions'
// angles, with each head's norm ahead of it where a call has one, to a tensor or to
// the token's cache slot (rope.cu, norm.cu).
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
#pragma once

#include <algorithm>
#include <type_traits>

#include "cache.cuh"

namespace sv {

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
    // the norm of each head (template NORM)
    const void* w[2];  // of q and k: D factors, or none
    int w_dtype;
    float eps;
};

// norm_e4m3.cu: norms on the way into an 8-bit cache (translation units of their own, to be compiled
// side by side)
cudaError_t launch_norm_e4m3(const RotArgs& A, int dtype, cudaStream_t st);

namespace {

// Whether a call has more than the rotation (spec_norm_rope, spec_norm_kv_write): each
// head of q and k is divided by the root of its mean square and multiplied by the
// weights first, and keys can go to a tensor besides their slot.
constexpr bool PLAIN = false, NORM = true;

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

constexpr int MAX_ROW = 256;  // channels of a head, at most
__device__ __forceinline__ void load_weights(const RotArgs& A, float* to) {
    for (int i = threadIdx.x; i < 2 * MAX_ROW; i += ROT_THREADS) {
        const int side = i / MAX_ROW, d = i % MAX_ROW;
        const void* w = side ? A.w[1] : A.w[0];
        float f = 1.f;
        if (w && d < A.D)
            f = A.w_dtype == SPEC_F32    ? static_cast<const float*>(w)[d]
                : A.w_dtype == SPEC_BF16 ? to_f32(static_cast<const __nv_bfloat16*>(w)[d])
                                         : to_f32(static_cast<const __half*>(w)[d]);
        to[i] = f;
    }
}

// T: element type of the tensors; VEC: elements of a vector; IP: lanes of a
// token; E4: the cache is e4m3 (else of type T); PAIR: half layout (else
// interleaved, or nothing turns); N: with the norm.
template <typename T, int VEC, int IP, bool E4, bool PAIR, bool N>
__global__ void __launch_bounds__(ROT_THREADS, N ? 2 : 3) k_rotate(const __grid_constant__ RotArgs A) {
    begin_after_previous();
    // weights of q and k as float32
    __shared__ __align__(16) float weights[N ? 2 * MAX_ROW : 4];
    if constexpr (N) {
        load_weights(A, weights);
        __syncthreads();
    }
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

    const float inv_d = N ? 1.f / float(A.D) : 0.f;
    // With a norm: weights and angles of this lane's item in one factor each, two side by side (what a head costs
    // in instructions bounds the kernel: with the weights read for each head, 32771 tokens took 129 us).
    // Half layout: y_a = fac0 a + fac1 b, y_b = fac2 a + fac3 b; else y = fac0 x + fac1 (x, the pair's exchanged).
    // Where nothing turns fac1 is 0, and the pair's other channel, which may be infinite, is masked to 0 (2% of
    // the time of pairs side by side; a choice made for each head or by a branch for infinite ones took 4 to 6).
    const uint32_t other_bits = pt.turns ? ~0u : 0u;
    auto masked = [&](float f) { return __uint_as_float(__float_as_uint(f) & other_bits); };
    uint64_t fac[N ? (PAIR ? 2 * VEC : VEC) : 1];
    auto factors = [&](int kind) {
        if constexpr (N) {
            const Place& p = hr ? pt : pp;
            const float* w = weights + kind * MAX_ROW + (p.on ? p.off : 0);
            const int second = p.on ? p.second : 0;
#pragma unroll
            for (int e = 0; e < VEC / 2; ++e) {
                const float w0 = w[2 * e], w1 = w[2 * e + 1];
                const bool turns = hr && p.turns;
                if constexpr (PAIR) {
                    const float c0 = turns ? cs[2 * e] : 1.f, c1 = turns ? cs[2 * e + 1] : 1.f;
                    const float s0 = turns ? sn[2 * e] : 0.f, s1 = turns ? sn[2 * e + 1] : 0.f;
                    const float v0 = w[second + 2 * e], v1 = w[second + 2 * e + 1];
                    fac[e] = f2_pack(w0 * c0, w1 * c1);
                    fac[VEC / 2 + e] = f2_pack(-v0 * s0, -v1 * s1);
                    fac[VEC + e] = f2_pack(w0 * s0, w1 * s1);
                    fac[VEC * 3 / 2 + e] = f2_pack(v0 * c0, v1 * c1);
                } else {
                    const float c = turns ? cs[e] : 1.f, s = turns ? sn[e] : 0.f;
                    fac[e] = f2_pack(w0 * c, w1 * c);
                    fac[VEC / 2 + e] = f2_pack(-w1 * s, w0 * s);
                }
            }
        }
    };
    // UH heads from h on: to `out`, or (bytes, scales) as e4m3, and to `also`; `w`: weights
    auto put = [&](int h, int hi, const Place& p, T* out, long long oh, uint8_t* bytes, uint8_t* scales,
                   const float* w = nullptr, T* also = nullptr, long long ah = 0) {
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
            if (N && w) {
                uint64_t a2[VEC / 2], b2[PAIR ? VEC / 2 : 1], sq = f2_pack(0.f, 0.f);
#pragma unroll
                for (int e = 0; e < VEC / 2; ++e) {
                    a2[e] = f2_pack(va[2 * e], va[2 * e + 1]);
                    sq = f2_fma(a2[e], a2[e], sq);
                    if constexpr (PAIR) {
                        b2[e] = p.second ? f2_pack(vb[2 * e], vb[2 * e + 1]) : f2_pack(0.f, 0.f);
                        sq = f2_fma(b2[e], b2[e], sq);
                    }
                }
                float s0, s1;
                f2_unpack(sq, s0, s1);
                float ss = p.on ? s0 + s1 : 0.f;
#pragma unroll
                for (int o = IP / 2; o; o >>= 1) ss += __shfl_xor_sync(gmask, ss, o, IP);
                const float f = rsqrtf(fmaf(ss, inv_d, A.eps));
                const uint64_t ff = f2_pack(f, f);
#pragma unroll
                for (int e = 0; e < VEC / 2; ++e) {
                    if constexpr (PAIR) {
                        f2_unpack(f2_mul(ff, f2_fma(fac[e], a2[e], f2_mul(fac[VEC / 2 + e], b2[e]))), va[2 * e], va[2 * e + 1]);
                        f2_unpack(f2_mul(ff, f2_fma(fac[VEC + e], a2[e], f2_mul(fac[VEC * 3 / 2 + e], b2[e]))), vb[2 * e], vb[2 * e + 1]);
                    } else {
                        const uint64_t other = f2_pack(masked(va[2 * e + 1]), masked(va[2 * e]));
                        f2_unpack(f2_mul(ff, f2_fma(fac[e], a2[e], f2_mul(fac[VEC / 2 + e], other))), va[2 * e], va[2 * e + 1]);
                    }
                }
            } else
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
                if (!N || !also) continue;
            }
            if (p.on) {
                Words<T, VEC> a, b;
#pragma unroll
                for (int e = 0; e < VEC / 2; ++e) {
                    set2(a, e, va[2 * e], va[2 * e + 1]);
                    if constexpr (PAIR) set2(b, e, vb[2 * e], vb[2 * e + 1]);
                    else set2(b, e, 0.f, 0.f);
                }
                auto store = [&](T* at) {
                    *reinterpret_cast<Words<T, VEC>*>(at) = a;
                    if (PAIR && p.second) *reinterpret_cast<Words<T, VEC>*>(at + p.second) = b;
                };
                if (!N || out) store(out + (h + u) * oh + p.off);
                if (N && also) store(also + (h + u) * ah + p.off);
            }
        }
    };
    // the tensor `kind`: f(its heads, an item's place, where they go)
    auto with = [&](int kind, auto&& f) {
        bool cached = A.slots && kind;
        const Heads& X = tensor(kind);
        if (cached && sr.row < 0) {
            if (!N || !X.out) return;
            cached = false;  // no slot, but a tensor
        }
        const Place p = kind != 2 && hr ? pt : pp;
        T* out = cached ? static_cast<T*>(kind == 1 ? A.c.k : A.c.v) + (E4 ? 0 : sr.row)
                        : static_cast<T*>(X.out) + t * X.ot;
        uint8_t* bytes = E4 && cached ? static_cast<uint8_t*>(kind == 1 ? A.c.k : A.c.v) + sr.row : nullptr;
        if (N && bytes) out = nullptr;
        f(X, p, out, cached ? A.c.head_stride : X.oh, bytes,
          E4 && cached ? (kind == 1 ? A.c.ks : A.c.vs) + sr.scale : nullptr,
          N && kind < 2 && A.eps >= 0.f ? weights + kind * MAX_ROW : nullptr,
          N && cached && X.out ? static_cast<T*>(X.out) + t * X.ot : nullptr);
    };

    if constexpr (PAIR) {
#pragma unroll 1
        for (int k = 0; k < 3; ++k) {
            const int base = k == 0 ? 0 : k == 1 ? A.q.n : A.q.n + A.k.n;
            const int lo = max(h0 - base, 0), end = min(h1 - base, tensor(k).n);
            if (lo >= end) continue;
            with(k, [&](const Heads& X, const Place& p, T* out, long long oh, uint8_t* bytes, uint8_t* scales,
                        const float* w, T* also) {
                const T* in = static_cast<const T*>(X.in) + t * X.it + lo * X.ih + p.off;
                if (N && w) factors(k);
#pragma unroll 1
                for (int i = lo; i < end; i += UH) {
                    load(in, X.ih, p, end - i);
                    in += UH * X.ih;
                    put(i, end, p, out, oh, bytes, scales, w, also, X.oh);
                }
            });
        }
    } else {
        int made = -1;  // whose factors there are
#pragma unroll 1
        while (kind < 3) {
            with(kind, [&](const Heads& X, const Place& p, T* out, long long oh, uint8_t* bytes, uint8_t* scales,
                           const float* w, T* also) {
                if (N && w && made != kind) {
                    factors(kind);
                    made = kind;
                }
                put(h, hi, p, out, oh, bytes, scales, w, also, X.oh);
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
template <typename T, bool E4, bool N>
__global__ void __launch_bounds__(ROT_THREADS) k_rotate_any(const __grid_constant__ RotArgs A) {
    begin_after_previous();
    const int lane = threadIdx.x & 31, H = A.q.n + A.k.n + A.v.n, hr = A.half_rot;
    const long long w = blockIdx.x * (long long)(ROT_THREADS / 32) + (threadIdx.x >> 5);
    if (w >= A.T * H) return;
    const long long t = w / H;
    const int h = int(w - t * H), kind = h < A.q.n ? 0 : h < A.q.n + A.k.n ? 1 : 2;
    const int hh = kind == 0 ? h : kind == 1 ? h - A.q.n : h - A.q.n - A.k.n;
    const SlotRow sr = slot_row(A, t, lane == 0 && h == 0);
    const bool turning = kind != 2 && hr;
    const Heads& X = kind == 0 ? A.q : kind == 1 ? A.k : A.v;
    const bool placed = A.slots && kind, cached = placed && sr.row >= 0;
    const bool plain = N ? X.out != nullptr : !placed;  // to a tensor too
    if (!cached && !plain) return;
    const T* in = static_cast<const T*>(X.in) + t * X.it + hh * X.ih;
    const int pairs = turning ? hr : 0, rest = A.D - 2 * pairs;
    const int pos = turning ? A.pos[t] : 0;
    float f = 1.f;
    const void* wp = nullptr;
    if (N && kind != 2 && A.eps >= 0.f) {
        wp = kind ? A.w[1] : A.w[0];
        float ss = 0.f;
        for (int d = lane; d < A.D; d += 32) {
            const float z = to_f32(in[d]);
            ss = fmaf(z, z, ss);
        }
        f = rsqrtf(fmaf(warp_sum_f(ss), 1.f / float(A.D), A.eps));
    }
    auto value = [&](int d) {
        float z = to_f32(in[d]);
        if (N) {
            z *= f;
            if (wp)
                z *= A.w_dtype == SPEC_F32    ? static_cast<const float*>(wp)[d]
                     : A.w_dtype == SPEC_BF16 ? to_f32(static_cast<const __nv_bfloat16*>(wp)[d])
                                              : to_f32(static_cast<const __half*>(wp)[d]);
        }
        return z;
    };
    // item i: a pair's two values and channels, or one of the rest (second -1)
    auto get = [&](int i, int& a, int& b, float& x, float& y) {
        if (i < pairs) {
            a = A.interleaved ? 2 * i : i;
            b = A.interleaved ? a + 1 : i + hr;
            float c, s;
            angle(A.turns[i], pos, c, s);
            c *= A.scale;
            s *= A.scale * A.sign;
            const float u = value(a), v = value(b);
            x = u * c - v * s;
            y = u * s + v * c;
        } else {
            a = i + pairs;
            b = -1;
            x = value(a);
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
        } else if (cached) {
            T* out = static_cast<T*>(kind == 1 ? A.c.k : A.c.v) + sr.row + hh * A.c.head_stride;
            out[a] = from_f32<T>(x);
            if (b >= 0) out[b] = from_f32<T>(y);
        }
        if (plain) {
            T* out = static_cast<T*>(X.out) + t * X.ot + hh * X.oh;
            out[a] = from_f32<T>(x);
            if (b >= 0) out[b] = from_f32<T>(y);
        }
    }
}

// Lanes that a token's heads need at VEC elements a vector (more than 32: none);
// two vectors an item only where pairs are half a head apart.
int lanes_for(const RotArgs& A, int vec) {
    if (!A.half_rot || A.interleaved) return A.D / vec;
    return std::max(A.half_rot / vec + (A.D - 2 * A.half_rot) / vec, A.v.n ? (A.D / vec + 1) / 2 : 0);
}

template <typename T, int VEC, bool E4, bool PAIR, bool N>
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
    auto* kernel = ip == 4    ? k_rotate<T, VEC, 4, E4, PAIR, N>
                   : ip == 8  ? k_rotate<T, VEC, 8, E4, PAIR, N>
                   : ip == 16 ? k_rotate<T, VEC, 16, E4, PAIR, N>
                              : k_rotate<T, VEC, 32, E4, PAIR, N>;
    return launch_behind(kernel, grid, ROT_THREADS, 0, st, A);
}

template <typename T, bool E4, bool N>
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
        return side(A.q, true) && side(A.k, A.k.out != nullptr) && side(A.v, false);
    };
    const bool pair = A.half_rot && !A.interleaved;
    if constexpr (E4 && sizeof(T) == 2)  // bytes then go out 16 at a time too
        if (!pair && ok(16)) return launch_rotate<T, 16, E4, false, N>(A, st);
    if (ok(8)) return pair ? launch_rotate<T, 8, E4, true, N>(A, st) : launch_rotate<T, 8, E4, false, N>(A, st);
    if (ok(4)) return pair ? launch_rotate<T, 4, E4, true, N>(A, st) : launch_rotate<T, 4, E4, false, N>(A, st);
    const long long warps = A.T * (A.q.n + A.k.n + A.v.n), grid = (warps + ROT_THREADS / 32 - 1) / (ROT_THREADS / 32);
    if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
    return launch_behind(k_rotate_any<T, E4, N>, dim3(unsigned(grid)), ROT_THREADS, 0, st, A);
}

inline spec_status check_table(const spec_rope_table* t, int D) {
    if (!t->turns || t->rot < 2 || t->rot > D || t->rot % 2) return SPEC_ERR_INVALID_ARG;
    if (t->layout != SPEC_ROPE_HALF && t->layout != SPEC_ROPE_INTERLEAVED)
        return SPEC_ERR_INVALID_ARG;
    if (!aligned(t->turns, 8)) return SPEC_ERR_UNSUPPORTED;
    return SPEC_OK;
}

}  // namespace
}  // namespace sv
