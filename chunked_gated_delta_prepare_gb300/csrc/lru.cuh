// What the forward, the gradient and the single-token form of the gated linear recurrence share.
//
//   h_t = a_t h_{t-1} + s_t g_t x_t,   q = sigmoid(r_t), g = sigmoid(i_t) (1 without i)
//   RATE:  a = e^{-k q}, k = c softplus(lam), s = sqrt(1 - a^2);     else  a = q, s = 1 - a
//
// A thread takes two neighbouring channels through the packed fp32 instructions.
#pragma once

#include <algorithm>
#include <type_traits>

#include "layer_common.cuh"
#include "layer_internal.h"

namespace gdr {
namespace layer {

// A tile: 128 tokens of a sequence by 64 channels, 16 warps of 8 tokens each, two channels a lane.
constexpr int kLruTokens = 8, kLruWarps = 16, kLruTile = kLruTokens * kLruWarps, kLruCols = 64;
static_assert(kLruTile == kLruKept, "a kept state for each tile");

// The operator as the kernels take it.  RowTensor::vec: two neighbouring channels are one aligned access.
struct Lru {
    Seqs q;
    int D;
    int cols;                // blocks of channels
    RowTensor x, r, i;
    const float *lam, *h0;
    float c;
    bool vec;                // of contiguous tensors of tokens
};

// ex2.approx leans low near 1 (see ssm.cuh): the exponent of a decay leans up by as much.
constexpr float kLruLean = 8e-9f;

__device__ __forceinline__ F2 neg2(F2 v) { return v ^ 0x8000000080000000ull; }

template <typename IO> __device__ __forceinline__ RawN<IO, 2> load2(const IO* p, int left, bool vec) {
    RawN<IO, 2> r;
    if (vec && left >= 2) {
        if constexpr (sizeof(IO) == 4) *reinterpret_cast<uint2*>(&r) = __ldg(reinterpret_cast<const uint2*>(p));
        else *reinterpret_cast<uint32_t*>(&r) = __ldg(reinterpret_cast<const uint32_t*>(p));
    } else {
        r.e[0] = left > 0 ? p[0] : from_f<IO>(0.f);
        r.e[1] = left > 1 ? p[1] : from_f<IO>(0.f);
    }
    return r;
}
template <typename IO> __device__ __forceinline__ void store2(IO* p, F2 v, int left, bool vec) {
    const float2 f = unpack2(v);
    RawN<IO, 2> r;
    from_f2(r.e, f.x, f.y);
    if (vec && left >= 2) {
        if constexpr (sizeof(IO) == 4) *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(&r);
        else *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<const uint32_t*>(&r);
    } else {
        if (left > 0) p[0] = r.e[0];
        if (left > 1) p[1] = r.e[1];
    }
}
template <typename IO> __device__ __forceinline__ F2 wide2(const RawN<IO, 2>& r) {
    const float2 f = to_f2(r.e);
    return pack2(f.x, f.y);
}
// fp32 pairs of [.., D] that start anywhere; zeros without p or past the row.
__device__ __forceinline__ F2 state2(const float* p, int64_t at, int left) {
    return pack2(p && left > 0 ? p[at] : 0.f, p && left > 1 ? p[at + 1] : 0.f);
}
__device__ __forceinline__ void put_state2(float* p, int64_t at, F2 v, int left) {
    const float2 f = unpack2(v);
    if (left > 0) p[at] = f.x;
    if (left > 1) p[at + 1] = f.y;
}

// sigmoid(v) and 1 - sigmoid(v), both to relative accuracy: with e = e^-|v| <= 1 the smaller is e / (1 + e), the larger
// one less that.
__device__ __forceinline__ void sigmoid_both2(F2 v, F2& up, F2& down) {
    const float2 f = unpack2(v);
    const F2 e = pack2(ex2(-fabsf(f.x) * kLog2e), ex2(-fabsf(f.y) * kLog2e));
    const F2 small = mul2(e, rcp_2(add2(both(1.f), e))), large = add2(both(1.f), neg2(small));
    const float2 s = unpack2(small), l = unpack2(large);
    up = pack2(f.x < 0.f ? s.x : l.x, f.y < 0.f ? s.y : l.y);
    down = pack2(f.x < 0.f ? l.x : s.x, f.y < 0.f ? l.y : s.y);
}

// 1 - e^w for w <= 0, given e^(w/2) = a: 1 - a^2, and near 0, where that cancels, -w (1 + w/2 (1 + w/3 (...))): what follows
// w^5 / 720 is below 2^-24 of the sum at w = -1/4.
__device__ __forceinline__ F2 one_less(F2 w, F2 a) {
    F2 p = fma2(w, both(1.f / 6), both(1.f));
    p = fma2(mul2(w, p), both(1.f / 5), both(1.f));
    p = fma2(mul2(w, p), both(1.f / 4), both(1.f));
    p = fma2(mul2(w, p), both(1.f / 3), both(1.f));
    p = fma2(mul2(w, p), both(1.f / 2), both(1.f));
    const float2 near = unpack2(neg2(mul2(w, p))), far = unpack2(fma2(neg2(a), a, both(1.f))), at = unpack2(w);
    return pack2(at.x > -0.25f ? near.x : far.x, at.y > -0.25f ? near.y : far.y);
}

__device__ __forceinline__ float rsqrt_fast(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / sqrt(v): finite for 0, and NaN is left to what it multiplies.
__device__ __forceinline__ F2 rsqrt2(F2 v) {
    const float2 f = unpack2(v);
    return pack2(rsqrt_fast(fmaxf(f.x, 1e-37f)), rsqrt_fast(fmaxf(f.y, 1e-37f)));
}

// A channel pair's constants: k = c softplus(lam), and its slope c sigmoid(lam).
struct Rate {
    F2 k, slope;
};
__device__ __forceinline__ float rate_of(float lam, float c) {
    return c * (fmaxf(lam, 0.f) + log1pf(expf(-fabsf(lam))));     // a NaN comes through the logarithm
}
__device__ __forceinline__ Rate load_rate(const Lru& a, int ch, bool slope) {
    Rate o{0, 0};
    const float l0 = ch < a.D ? a.lam[ch] : 0.f, l1 = ch + 1 < a.D ? a.lam[ch + 1] : 0.f;
    o.k = pack2(rate_of(l0, a.c), rate_of(l1, a.c));
    if (slope) o.slope = pack2(a.c / (1.f + expf(-l0)), a.c / (1.f + expf(-l1)));
    return o;
}

// The decay alone.
template <bool RATE> __device__ __forceinline__ F2 decay_of(F2 r, const Rate& k) {
    F2 up, down;
    if (RATE) return ex2_2(fma2(mul2(k.k, both(-kLog2e)), sigmoid2(r), both(kLruLean)));
    sigmoid_both2(r, up, down);
    return up;
}
// The decay and the input's part s.
template <bool RATE> __device__ __forceinline__ void decay_and_part(F2 r, const Rate& k, F2& a, F2& s) {
    if (RATE) {
        const F2 kq = mul2(k.k, sigmoid2(r));
        a = ex2_2(fma2(kq, both(-kLog2e), both(kLruLean)));
        const F2 m = one_less(mul2(kq, both(-2.f)), a);
        s = mul2(m, rsqrt2(m));
    } else {
        sigmoid_both2(r, a, s);
    }
}

// A block's tile and channels.
struct LruTile {
    int seq;                 // -1: no such tile
    int64_t number;          // of the tile over all sequences
    int64_t first;           // its first token on the axis
    int len;                 // tokens, 0 of an empty sequence
    bool head, tail;         // the first, the last of its sequence
    int ch, left;            // the thread's first channel, and how many there are from it on
};
__device__ __forceinline__ LruTile lru_tile(const Lru& a, int64_t block) {
    LruTile t;
    t.number = block / a.cols;
    const int col = (int)(block - t.number * a.cols);
    const TileAt at = find_tile(a.q, t.number, kLruTile);
    t.seq = at.seq;
    t.first = at.start + at.tile * kLruTile;
    const int64_t rest = at.len - at.tile * kLruTile;
    t.len = (int)(rest < kLruTile ? rest : kLruTile);
    t.head = at.tile == 0;
    t.tail = rest <= kLruTile;
    t.ch = col * kLruCols + (threadIdx.x & 31) * 2;
    t.left = a.D - t.ch;
    return t;
}

// Calls f with a value of the io type and whether there are rates and input gates.
template <typename F> cudaError_t lru_types(int io, bool rate, bool gate, F f) {
    const auto forms = [&](auto v) {
        if (rate) return gate ? f(v, std::true_type(), std::true_type()) : f(v, std::true_type(), std::false_type());
        return gate ? f(v, std::false_type(), std::true_type()) : f(v, std::false_type(), std::false_type());
    };
    if (io == GDR_F32) return forms(float());
    if (io == GDR_BF16) return forms(__nv_bfloat16());
    return forms(__half());
}

inline bool lru_pairs(const void* p, int64_t ld, int64_t e) {
    return reinterpret_cast<uintptr_t>(p) % (2 * e) == 0 && ld % 2 == 0;
}
inline Lru lru_of(const LruArgs& a, const LruTensors& t) {
    const int64_t e = a.io == GDR_F32 ? 4 : 2;
    Lru k{};
    k.q = Seqs{a.cu, a.total, a.T, (int)a.n};
    k.D = a.D;
    k.cols = (a.D + kLruCols - 1) / kLruCols;
    k.x = t.x;
    k.r = t.r;
    k.i = t.i;
    for (RowTensor* v : {&k.x, &k.r, &k.i}) v->vec = lru_pairs(v->p, v->ld, e);
    k.lam = t.lam;
    k.h0 = t.h0;
    k.c = a.c;
    return k;
}

}  // namespace layer
}  // namespace gdr
