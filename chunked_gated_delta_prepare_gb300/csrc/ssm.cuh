// What the forward, the backward and the single-token form of the selective scan share.
//
//   h_t[d][n] = exp(Delta_t[d] A[d][n]) h_{t-1}[d][n] + Delta_t[d] x_t[d] B_t[g][n],   Delta = softplus(dt + bias)
//   y_t[d]    = (sum_n C_t[g][n] h_t[d][n] + Dk[d] x_t[d]) silu(z_t[d])
//
// A channel's states lie on LN neighbouring lanes, 4 on each (N <= 4 LN, the rest zero), a lane takes DC neighbouring
// channels.  Products go two channels at a time through the packed fp32 instructions: two independent fp32 operations
// each, rounded as alone.
#pragma once

#include "layer_common.cuh"
#include "layer_internal.h"

namespace gdr {
namespace layer {

constexpr int kSsmThreads = 128;

// exp(Delta A) is ex2 of a product: ex2.approx's error is below 2^-22 of the result, and its mean below 1e-8 near 1, where
// slow decays live.

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
    RowTensor x, dt, z, B, C;
    const float *A, *bias, *Dk, *h0;
    bool softplus;
    bool vec;                // rows of D elements on 16-byte boundaries in the contiguous tensors of tokens
};

// The channels of a block: [c0, end) of one group.
struct Channels {
    int group, c0, end;
};
__device__ __forceinline__ Channels block_channels(const Ssm& a, int width) {
    const int blocks = (a.per + width - 1) / width;
    Channels c;
    c.group = blockIdx.y / blocks;
    c.c0 = c.group * a.per + (blockIdx.y - c.group * blocks) * width;
    c.end = (c.group + 1) * a.per;
    return c;
}

// 8 channels from c of a token's row; `left` of them exist.
template <typename IO> __device__ __forceinline__ Raw8<IO> load_row8(const RowTensor& t, int64_t row, int c, int left) {
    return load8(reinterpret_cast<const IO*>(t.p) + row * t.ld + c, left, t.vec && (c & 7) == 0);
}

__device__ __forceinline__ float step_size(const Ssm& a, float raw, int c) {
    if (a.bias) raw += a.bias[c];
    return a.softplus ? softplus(raw) : raw;
}

// log2(e) A of channels c .. c + DC and states n .. n + 4, channel pairs packed; zero outside.
template <int DC>
__device__ __forceinline__ void load_decay(const Ssm& a, int c, int end, int n, F2 (&A2)[4][DC / 2]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < DC / 2; ++i) {
            float v[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int d = c + 2 * i + k;
                v[k] = d < end && n + j < a.N ? a.A[(int64_t)d * a.N + n + j] * kLog2e : 0.f;
            }
            A2[j][i] = pack2(v[0], v[1]);
        }
}

// States [d][n] of channels c .. c + DC and states n .. n + 4, to and from memory [D][N].
template <int DC>
__device__ __forceinline__ void load_states(const float* p, const Ssm& a, int c, int end, int n, F2 (&h)[4][DC / 2]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < DC / 2; ++i) {
            float v[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int d = c + 2 * i + k;
                v[k] = p && d < end && n + j < a.N ? p[(int64_t)d * a.N + n + j] : 0.f;
            }
            h[j][i] = pack2(v[0], v[1]);
        }
}
template <int DC>
__device__ __forceinline__ void store_states(float* p, const Ssm& a, int c, int end, int n, const F2 (&h)[4][DC / 2]) {
#pragma unroll
    for (int i = 0; i < DC; ++i) {
        if (c + i >= end) continue;
        float* q = p + (int64_t)(c + i) * a.N + n;
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = i & 1 ? unpack2(h[j][i / 2]).y : unpack2(h[j][i / 2]).x;
        if (n + 4 <= a.N && (reinterpret_cast<uintptr_t>(q) & 15) == 0) {
            *reinterpret_cast<float4*>(q) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + j < a.N) q[j] = v[j];
        }
    }
}

// B and C of `tokens` tokens from `row`, each value twice (for both halves of a packed product): [t][4 LN][2].
// Tokens from `live` on read as zero.
template <typename IO, int LN>
__device__ __forceinline__ void load_bc(const Ssm& a, const RowTensor& t, int group, int64_t row, int live, int tokens,
                                        float2* out) {
    for (int i = threadIdx.x; i < tokens * 4 * LN; i += kSsmThreads) {
        const int k = i / (4 * LN), n = i % (4 * LN);
        const float v =
            k < live && n < a.N ? to_f(reinterpret_cast<const IO*>(t.p)[(row + k) * t.ld + group * a.N + n]) : 0.f;
        out[i] = make_float2(v, v);
    }
}

// Sums over a channel's LN lanes of v[0 .. DC), one for each of DC channels: lane q < DC is left with the sum of channel
// kept<DC>(q) in v[0].  Partners halve the channels between them while there is more than one.
template <int DC> __device__ __forceinline__ int kept(int q) { return DC == 2 ? q & 1 : (q & 1) * 2 + (q >> 1 & 1); }
template <int LN, int DC> __device__ __forceinline__ void lanes_sum(float (&v)[DC], int q) {
    static_assert(LN >= DC, "a lane for each channel");
#pragma unroll
    for (int size = DC / 2, m = 1; m < LN; size /= 2, m *= 2) {
        if (size == 0) {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], m);
        } else {
            const bool up = q & m;
#pragma unroll
            for (int i = 0; i < DC / 2; ++i) {
                if (i >= size) break;
                const float give = up ? v[i] : v[i + size], keep = up ? v[i + size] : v[i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, give, m);
            }
        }
    }
}

// Calls f with a value of the io type and the lanes of a channel.
template <typename F> cudaError_t ssm_types(int io, int N, F f) {
    const auto lanes = [&](auto v) {
        if (N <= 8) return f(v, std::integral_constant<int, 2>());
        if (N <= 16) return f(v, std::integral_constant<int, 4>());
        if (N <= 32) return f(v, std::integral_constant<int, 8>());
        return f(v, std::integral_constant<int, 16>());
    };
    if (io == GDR_F32) return lanes(float());
    if (io == GDR_BF16) return lanes(__nv_bfloat16());
    return lanes(__half());
}

inline int ssm_lanes(int64_t N) { return N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }

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
