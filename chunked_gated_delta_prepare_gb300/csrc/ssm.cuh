// What the forward, the backward and the single-token form of the selective scan share.
//
//   h_t[d][n] = exp(Delta_t[d] A[d][n]) h_{t-1}[d][n] + Delta_t[d] x_t[d] B_t[g][n],   Delta = softplus(dt + bias)
//   y_t[d]    = (sum_n C_t[g][n] h_t[d][n] + Dk[d] x_t[d]) silu(z_t[d])
//
// A channel's states lie on LN neighbouring lanes, NS (4 or 8) on each, the rest zero; a lane takes DC neighbouring
// channels.  Products go two states at a time through the packed fp32 instructions: two independent fp32 operations
// each, rounded as alone.
#pragma once

#include "layer_common.cuh"
#include "layer_internal.h"

namespace gdr {
namespace layer {

// exp(Delta A), A2 = log2(e) A.  ex2.approx is good to 2^-22 of its result, but leans low: near 1, where the slow decays
// live, by 5e-9 on average (measured for exponents of -2^-9 .. -2^-14).  A state that keeps a thousand tokens would add
// that up to 5e-6 of itself, so the exponent leans up by as much; the sum rides on the product's own instruction.
constexpr float kLean = 8e-9f;
__device__ __forceinline__ F2 decay2(F2 A2, F2 d) { return ex2_2(fma2(A2, d, both(kLean))); }
__device__ __forceinline__ float decay(float A2, float d) { return ex2(fmaf(A2, d, kLean)); }

// log(1 + e^x) = max(x, 0) + log(1 + e), e = e^-|x| in (0, 1].  log(1 + e) = 2 atanh(r), r = e / (2 + e) <= 1/3, by its
// series to r^13 (what follows is below 2^-23 of the sum): relative accuracy also where e is small, as steps of 0.001
// need it, at half the instructions of log1pf.
__device__ __forceinline__ F2 softplus2(F2 x) {
    const float2 f = unpack2(x);
    const F2 e = ex2_2(mul2(pack2(fminf(f.x, -f.x), fminf(f.y, -f.y)), both(kLog2e)));
    const F2 r = mul2(e, rcp_2(add2(both(2.f), e))), t = mul2(r, r);
    F2 s = fma2(t, both(1.f / 13), both(1.f / 11));
    s = fma2(s, t, both(1.f / 9));
    s = fma2(s, t, both(1.f / 7));
    s = fma2(s, t, both(1.f / 5));
    s = fma2(s, t, both(1.f / 3));
    s = fma2(s, t, both(1.f));
    return fma2(add2(r, r), s, pack2(fmaxf(f.x, 0.f), fmaxf(f.y, 0.f)));      // a NaN comes through r
}
__device__ __forceinline__ float softplus(float x) { return unpack2(softplus2(both(x))).x; }

// The operator as the kernels take it.
struct Ssm {
    Seqs q;
    int D, N, G, per;        // per = D / G channels share the B and C of a group
    int seg;                 // tokens of a segment
    int first_seq;           // ssm_join: sequence of the grid's first row
    RowTensor x, dt, z, B, C;
    const float *A, *bias, *Dk, *h0;
    bool softplus;
    bool vec;                // rows of D elements on 16-byte boundaries in the contiguous tensors of tokens
};

// The channels of a block: [c0, end) of one group.
struct Channels {
    int group, block, c0, end;
};
__device__ __forceinline__ Channels block_channels(const Ssm& a, int width) {
    const int blocks = (a.per + width - 1) / width;
    Channels c;
    c.group = blockIdx.y / blocks;
    c.block = blockIdx.y - c.group * blocks;
    c.c0 = c.group * a.per + c.block * width;
    c.end = (c.group + 1) * a.per;
    return c;
}

__device__ __forceinline__ float step_size(const Ssm& a, float raw, int c) {
    if (a.bias) raw += a.bias[c];
    return a.softplus ? softplus(raw) : raw;
}

// NS states from n of channels c .. c + DC, to and from memory [D][N], neighbours packed; zero outside.
template <int DC, int NS>
__device__ __forceinline__ void load_states(const float* p, const Ssm& a, int c, int end, int n, F2 (&h)[DC][NS / 2]) {
#pragma unroll
    for (int i = 0; i < DC; ++i) {
        const float* q = p + (int64_t)(c + i) * a.N + n;
        float v[NS];
#pragma unroll
        for (int j = 0; j < NS; j += 4) {
            if (p && c + i < end && n + j + 4 <= a.N && (reinterpret_cast<uintptr_t>(q) & 15) == 0) {
                const float4 f = *reinterpret_cast<const float4*>(q + j);
                v[j] = f.x, v[j + 1] = f.y, v[j + 2] = f.z, v[j + 3] = f.w;
            } else {
#pragma unroll
                for (int k = j; k < j + 4; ++k) v[k] = p && c + i < end && n + k < a.N ? q[k] : 0.f;
            }
        }
#pragma unroll
        for (int j = 0; j < NS / 2; ++j) h[i][j] = pack2(v[2 * j], v[2 * j + 1]);
    }
}
template <int DC, int NS>
__device__ __forceinline__ void store_states(float* p, const Ssm& a, int c, int end, int n, const F2 (&h)[DC][NS / 2]) {
#pragma unroll
    for (int i = 0; i < DC; ++i) {
        if (c + i >= end) continue;
        float* q = p + (int64_t)(c + i) * a.N + n;
#pragma unroll
        for (int j = 0; j < NS; j += 4) {
            const float2 lo = unpack2(h[i][j / 2]), hi = unpack2(h[i][j / 2 + 1]);
            if (n + j + 4 <= a.N && (reinterpret_cast<uintptr_t>(q) & 15) == 0) {
                *reinterpret_cast<float4*>(q + j) = make_float4(lo.x, lo.y, hi.x, hi.y);
            } else {
                const float v[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (n + j + k < a.N) q[j + k] = v[k];
            }
        }
    }
}

// log2(e) A of the same channels and states.
template <int DC, int NS>
__device__ __forceinline__ void load_decay(const Ssm& a, int c, int end, int n, F2 (&A2)[DC][NS / 2]) {
    load_states<DC, NS>(a.A, a, c, end, n, A2);
#pragma unroll
    for (int i = 0; i < DC; ++i)
#pragma unroll
        for (int j = 0; j < NS / 2; ++j) A2[i][j] = mul2(A2[i][j], both(kLog2e));
}

// Joins the segments of each sequence, in place.  ends: what a segment leaves from a zero state (first_whole: the first
// one from h0) becomes the state before it, h0 before the first.  dends (may be nullptr): the gradient that a segment's
// tokens send to the state before it becomes the gradient of the state after it, dh_final after the last.  sums: a
// segment's sums of Delta.  Sequences of one segment are left alone.
cudaError_t ssm_join(const Ssm& a, float* ends, float* dends, const float* sums, const float* dh_final, bool first_whole,
                     cudaStream_t s);

// Calls f with a value of the io type and the lanes of a channel, NS states on each.
template <int NS, typename F> cudaError_t ssm_types(int io, int N, F f) {
    const auto lanes = [&](auto v) {
        if (N <= 8) return f(v, std::integral_constant<int, 8 / NS>());
        if (N <= 16) return f(v, std::integral_constant<int, 16 / NS>());
        if (N <= 32) return f(v, std::integral_constant<int, 32 / NS>());
        return f(v, std::integral_constant<int, 64 / NS>());
    };
    if (io == GDR_F32) return lanes(float());
    if (io == GDR_BF16) return lanes(__nv_bfloat16());
    return lanes(__half());
}

inline int ssm_lanes(int64_t N, int NS) { return (N <= 8 ? 8 : N <= 16 ? 16 : N <= 32 ? 32 : 64) / NS; }

// Blocks of `width` channels in all groups.
inline int64_t ssm_blocks(const SsmArgs& a, int width) { return a.G * ((int64_t)(a.D / a.G + width - 1) / width); }

inline Ssm ssm_of(const SsmArgs& a, const SsmTensors& t) {
    Ssm k{};
    k.q = Seqs{a.cu, a.total, a.T, (int)a.n};
    k.D = a.D;
    k.N = a.N;
    k.G = a.G;
    k.per = a.D / a.G;
    k.x = t.x;
    k.dt = t.dt;
    k.z = t.z;
    k.B = t.B;
    k.C = t.C;
    k.A = t.A;
    k.bias = t.bias;
    k.Dk = t.Dk;
    k.h0 = t.h0;
    k.softplus = a.softplus;
    return k;
}

}  // namespace layer
}  // namespace gdr
