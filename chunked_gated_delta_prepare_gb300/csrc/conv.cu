// The short causal convolution of each channel over its own tokens, its gradient, and its single-token form.
//
//   p_t = b + sum_{j < W} w_j x_{t - W + 1 + j},   y_t = silu(p_t) or p_t;   x before the sequence: the W - 1 rows of
//   its state, or zero.  The state it leaves is the last W - 1 inputs.
//
// Bound: memory, x read once and y written once.  A thread takes neighbouring channels (8 of them, one 16-byte load of
// a 16-bit type) down a run of tokens with the window of W inputs in registers, so each input is loaded once and the
// next 8 loads are in flight while the last ones are used; only the W - 1 inputs before a run are read again.
//
// Gradient: with dp_t = dy_t act'(p_t), p_t formed again from x,
//   dx_u = sum_j w_j dp_{u + W - 1 - j},  dw_j = sum_t dp_t x_{t - W + 1 + j},  db = sum_t dp_t.
// The same walk with a second window, of dp: at token t the gradient of x_{t - W + 1} is complete.  A run goes W - 1
// tokens past its end for the last of its dx.  4 channels a thread here: two windows, w and the sums of dw take 18
// registers a channel, and 8 channels left two blocks an SM.  dw and db are added in registers, then over the block's
// runs in shared memory, and leave as one row of partial sums a block, which column_sum adds in a fixed order.
#include <algorithm>

#include "layer_common.cuh"
#include "layer_internal.h"

namespace gdr {
namespace layer {
namespace {

constexpr int kThreads = 128;
constexpr int kForwardRun = 16, kBackwardRun = 32;   // tokens of a thread

// Lanes that share a token: the vectors of a row, at most 32 (a block's threads then hold kThreads / lanes runs).
int row_lanes(int64_t D, int channels) {
    int l = 1;
    while (l < 32 && l * channels < D) l *= 2;
    return l;
}

struct Conv {
    Seqs q;
    int64_t D;
    RowTensor x;
    const void *w, *b, *state;
    int lanes;       // row_lanes
    bool silu;
    bool vec;        // rows of D elements on 16-byte boundaries in every contiguous tensor
};

// Input u of a sequence: a token (u >= 0), a row of its state, or zero.
template <int N, typename IO>
__device__ __forceinline__ RawN<IO, N> input_at(const Conv& a, int seq, int64_t start, int64_t u, int64_t c, int back) {
    const int64_t left = a.D - c;
    if (u >= 0) return load_n<N>(reinterpret_cast<const IO*>(a.x.p) + (start + u) * a.x.ld + c, left, a.x.vec);
    if (a.state)
        return load_n<N>(reinterpret_cast<const IO*>(a.state) + ((int64_t)seq * back + back + u) * a.D + c, left, a.vec);
    return load_n<N>((const IO*)nullptr, 0, false);
}

// w[j][i]: tap j of channel c + i
template <int N, int W, typename IO>
__device__ __forceinline__ void load_taps(const Conv& a, int64_t c, float (&w)[W][N], float (&b)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const bool in = c + i < a.D;
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = in ? to_f(reinterpret_cast<const IO*>(a.w)[(c + i) * W + j]) : 0.f;
        b[i] = in && a.b ? to_f(reinterpret_cast<const IO*>(a.b)[c + i]) : 0.f;
    }
}

template <typename IO, int W>
__global__ void __launch_bounds__(kThreads) conv_forward_kernel(Conv a, IO* __restrict__ y, IO* __restrict__ state_out) {
    constexpr int N = 8, kBack = W - 1, U = 8;
    const int lane = threadIdx.x % a.lanes, sub = threadIdx.x / a.lanes;
    const int tile = kForwardRun * (kThreads / a.lanes);
    const int64_t c = ((int64_t)blockIdx.y * a.lanes + lane) * N, left = a.D - c;
    const TileAt at = find_tile(a.q, blockIdx.x, tile);
    const int64_t t0 = at.tile * tile + (int64_t)sub * kForwardRun;
    if (at.seq < 0 || left <= 0 || (t0 >= at.len && t0 > 0)) return;

    float win[W][N], w[W][N], b[N];
    load_taps<N, W, IO>(a, c, w, b);
#pragma unroll
    for (int j = 0; j < kBack; ++j) widen(input_at<N, IO>(a, at.seq, at.start, t0 - kBack + j, c, kBack), win[j]);

    const IO* xp = reinterpret_cast<const IO*>(a.x.p) + (at.start + t0) * a.x.ld + c;
    IO* yp = y + (at.start + t0) * a.D + c;
    const int run = (int)min((int64_t)kForwardRun, at.len - t0);
    for (int i0 = 0; i0 < run; i0 += U) {
        RawN<IO, N> raw[U];
#pragma unroll
        for (int i = 0; i < U; ++i) raw[i] = load_n<N>(xp + (i0 + i) * a.x.ld, i0 + i < run ? left : 0, a.x.vec);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            widen(raw[i], win[kBack]);
            float o[N];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                o[k] = b[k];
#pragma unroll
                for (int j = 0; j < W; ++j) o[k] = fmaf(w[j][k], win[j][k], o[k]);
                if (a.silu) o[k] *= sigmoid(o[k]);
#pragma unroll
                for (int j = 0; j < kBack; ++j) win[j][k] = win[j + 1][k];
            }
            store_n(yp + (i0 + i) * a.D, o, i0 + i < run ? left : 0, a.vec);
        }
    }
    if (t0 == 0 && state_out)                 // the first run leaves the state, an empty sequence's too
#pragma unroll
        for (int j = 0; j < kBack; ++j)
            store_raw(state_out + ((int64_t)at.seq * kBack + j) * a.D + c,
                      input_at<N, IO>(a, at.seq, at.start, at.len - kBack + j, c, kBack), left, a.vec);
}

template <typename IO, int W>
__global__ void __launch_bounds__(kThreads)
conv_backward_kernel(Conv a, const IO* __restrict__ dy, const IO* __restrict__ d_state_out, IO* __restrict__ dx,
                     IO* __restrict__ d_state, float* __restrict__ partial) {
    constexpr int N = 4, kBack = W - 1, U = 4;
    __shared__ float sums[kThreads][N * (W + 1) + 1];     // + 1: threads on different banks
    const int lane = threadIdx.x % a.lanes, sub = threadIdx.x / a.lanes, subs = kThreads / a.lanes;
    const int tile = kBackwardRun * subs;
    const int64_t c = ((int64_t)blockIdx.y * a.lanes + lane) * N, left = a.D - c;
    const TileAt at = find_tile(a.q, blockIdx.x, tile);
    const int64_t t0 = at.tile * tile + (int64_t)sub * kBackwardRun;

    float dw[W][N], db[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        db[k] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][k] = 0.f;
    }
    if (at.seq >= 0 && left > 0 && (t0 < at.len || t0 == 0)) {
        float win[W][N], dp[W][N], w[W][N], b[N];
        load_taps<N, W, IO>(a, c, w, b);
#pragma unroll
        for (int j = 0; j < kBack; ++j) {
            widen(input_at<N, IO>(a, at.seq, at.start, t0 - kBack + j, c, kBack), win[j]);
#pragma unroll
            for (int k = 0; k < N; ++k) dp[j][k] = 0.f;
        }
        const int64_t t1 = min(t0 + kBackwardRun, at.len);
        // token t gives dp_t and completes dx_u, u = t - kBack, for u in [t0, t1); the first run has the state's
        // rows, u < 0, too
        for (int64_t s0 = t0; s0 < t1 + kBack; s0 += U) {
            RawN<IO, N> xr[U], yr[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const bool in = s0 + i < min(t1 + kBack, at.len);
                xr[i] = load_n<N>(reinterpret_cast<const IO*>(a.x.p) + (at.start + s0 + i) * a.x.ld + c, in ? left : 0,
                                  a.x.vec);
                yr[i] = load_n<N>(dy + (at.start + s0 + i) * a.D + c, in ? left : 0, a.vec);
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int64_t t = s0 + i, u = t - kBack;
                float g[N], o[N];
                widen(xr[i], win[kBack]);
                widen(yr[i], g);
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    if (a.silu) {
                        float p = b[k];
#pragma unroll
                        for (int j = 0; j < W; ++j) p = fmaf(w[j][k], win[j][k], p);
                        const float s = sigmoid(p);
                        g[k] *= s * fmaf(p, 1.f - s, 1.f);
                    }
                    // past the sequence dy is zero; what lies there times an infinite derivative must not count
                    if (t >= at.len) g[k] = 0.f;
                    dp[kBack][k] = g[k];
                    if (t < t1) {
                        db[k] += g[k];
#pragma unroll
                        for (int j = 0; j < W; ++j) dw[j][k] = fmaf(g[k], win[j][k], dw[j][k]);
                    }
                    o[k] = 0.f;
#pragma unroll
                    for (int j = 0; j < W; ++j) o[k] = fmaf(w[j][k], dp[kBack - j][k], o[k]);
#pragma unroll
                    for (int j = 0; j < kBack; ++j) win[j][k] = win[j + 1][k], dp[j][k] = dp[j + 1][k];
                }
                if (u >= t1 || (u < t0 && !(t0 == 0 && d_state))) continue;
                const int64_t row = u - (at.len - kBack);          // the row of the state it left, if it is one
                if (d_state_out && row >= 0) {
                    float e[N];
                    widen(load_n<N>(d_state_out + ((int64_t)at.seq * kBack + row) * a.D + c, left, a.vec), e);
#pragma unroll
                    for (int k = 0; k < N; ++k) o[k] += e[k];
                }
                if (u >= 0) store_n(dx + (at.start + u) * a.D + c, o, left, a.vec);
                else store_n(d_state + ((int64_t)at.seq * kBack + kBack + u) * a.D + c, o, left, a.vec);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
#pragma unroll
        for (int j = 0; j < W; ++j) sums[threadIdx.x][k * W + j] = dw[j][k];
        sums[threadIdx.x][N * W + k] = db[k];
    }
    __syncthreads();
    float* mine = partial + (int64_t)blockIdx.x * a.D * (W + 1);
    for (int i = threadIdx.x; i < a.lanes * N * (W + 1); i += kThreads) {
        const bool bias = i >= a.lanes * N * W;
        const int e = bias ? i - a.lanes * N * W : i, per = bias ? N : N * W;
        const int l = e / per, k = e % per;
        float s = 0.f;
        for (int r = 0; r < subs; ++r) s += sums[r * a.lanes + l][(bias ? N * W : 0) + k];
        const int64_t first = (int64_t)blockIdx.y * a.lanes * per + e;
        if (first < (bias ? a.D : a.D * W)) mine[(bias ? a.D * W : 0) + first] = s;
    }
}

template <typename IO, int W>
__global__ void __launch_bounds__(kThreads)
conv_step_kernel(Conv a, int64_t pool, const int* __restrict__ slots, IO* __restrict__ state, IO* __restrict__ y) {
    constexpr int N = 8, kBack = W - 1;
    const int64_t c = ((int64_t)blockIdx.y * kThreads + threadIdx.x) * N, left = a.D - c, row = blockIdx.x;
    if (left <= 0) return;
    const int64_t slot = slots ? slots[row] : row;
    float o[N];
    if (slot < 0 || slot >= pool) {
#pragma unroll
        for (int k = 0; k < N; ++k) o[k] = 0.f;
        store_n(y + row * a.D + c, o, left, a.vec);
        return;
    }
    RawN<IO, N> in[W];
#pragma unroll
    for (int j = 0; j < kBack; ++j) {     // plain loads: the state is written below
        const IO* p = state + (slot * kBack + j) * a.D + c;
        if (a.vec && left >= N) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(in[0]) / 16; ++i)
                reinterpret_cast<uint4*>(&in[j])[i] = reinterpret_cast<const uint4*>(p)[i];
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) in[j].e[i] = i < left ? p[i] : from_f<IO>(0.f);
        }
    }
    in[kBack] = load_n<N>(reinterpret_cast<const IO*>(a.x.p) + row * a.x.ld + c, left, a.x.vec);
    float w[W][N];
    load_taps<N, W, IO>(a, c, w, o);
#pragma unroll
    for (int k = 0; k < N; ++k) {
#pragma unroll
        for (int j = 0; j < W; ++j) o[k] = fmaf(w[j][k], to_f(in[j].e[k]), o[k]);
        if (a.silu) o[k] *= sigmoid(o[k]);
    }
    store_n(y + row * a.D + c, o, left, a.vec);
#pragma unroll
    for (int j = 0; j < kBack; ++j) store_raw(state + (slot * kBack + j) * a.D + c, in[j + 1], left, a.vec);
}

Conv conv_of(const ConvArgs& a, RowTensor x, const void* w, const void* b, const void* state,
             std::initializer_list<const void*> others) {
    Conv k{};
    k.q = Seqs{a.cu, a.total, a.T, (int)a.n};
    k.D = a.D;
    k.x = x;
    k.w = w;
    k.b = b;
    k.state = state;
    k.silu = a.silu;
    k.vec = a.D * (a.io == GDR_F32 ? 4 : 2) % 16 == 0 && reinterpret_cast<uintptr_t>(state) % 16 == 0;
    for (const void* p : others) k.vec = k.vec && reinterpret_cast<uintptr_t>(p) % 16 == 0;
    return k;
}

// Calls f with a value of the io type and the number of taps.
template <typename F> cudaError_t with_types(const ConvArgs& a, F f) {
    const auto taps = [&](auto io) {
        if (a.W == 2) return f(io, std::integral_constant<int, 2>());
        if (a.W == 3) return f(io, std::integral_constant<int, 3>());
        return f(io, std::integral_constant<int, 4>());
    };
    if (a.io == GDR_F32) return taps(float());
    if (a.io == GDR_BF16) return taps(__nv_bfloat16());
    return taps(__half());
}

unsigned channel_blocks(int64_t D, int lanes, int channels) {
    return (unsigned)((D + (int64_t)lanes * channels - 1) / ((int64_t)lanes * channels));
}

}  // namespace

cudaError_t conv_forward(const ConvArgs& a, RowTensor x, const void* w, const void* b, const void* state, void* y,
                         void* state_out, cudaStream_t s) {
    Conv k = conv_of(a, x, w, b, state, {y, state_out});
    k.lanes = row_lanes(a.D, 8);
    const int64_t tiles = tile_count(k.q, kForwardRun * (kThreads / k.lanes));
    return with_types(a, [&](auto io, auto taps) {
        using IO = decltype(io);
        conv_forward_kernel<IO, decltype(taps)::value>
            <<<dim3((unsigned)tiles, channel_blocks(a.D, k.lanes, 8)), kThreads, 0, s>>>(k, (IO*)y, (IO*)state_out);
        return cudaGetLastError();
    });
}

int64_t conv_partial_rows(const ConvArgs& a) {
    const Seqs q{a.cu, a.total, a.T, (int)a.n};
    return tile_count(q, kBackwardRun * (kThreads / row_lanes(a.D, 4)));
}

cudaError_t conv_backward(const ConvArgs& a, RowTensor x, const void* w, const void* b, const void* state,
                          const void* dy, const void* d_state_out, void* dx, float* dw, float* db, void* d_state,
                          float* partial, cudaStream_t s) {
    Conv k = conv_of(a, x, w, b, state, {dy, d_state_out, dx, d_state});
    k.lanes = row_lanes(a.D, 4);
    const int64_t tiles = conv_partial_rows(a);
    const cudaError_t e = with_types(a, [&](auto io, auto taps) {
        using IO = decltype(io);
        conv_backward_kernel<IO, decltype(taps)::value>
            <<<dim3((unsigned)tiles, channel_blocks(a.D, k.lanes, 4)), kThreads, 0, s>>>(
                k, (const IO*)dy, (const IO*)d_state_out, (IO*)dx, (IO*)d_state, partial);
        return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
    return column_sum(partial, tiles, a.D * (a.W + 1), a.D * a.W, dw, a.D, db, s);
}

cudaError_t conv_step(const ConvArgs& a, int64_t pool, const int* slots, RowTensor x, const void* w, const void* b,
                      void* state, void* y, cudaStream_t s) {
    const Conv k = conv_of(a, x, w, b, state, {y});
    return with_types(a, [&](auto io, auto taps) {
        using IO = decltype(io);
        conv_step_kernel<IO, decltype(taps)::value>
            <<<dim3((unsigned)a.n, channel_blocks(a.D, kThreads, 8)), kThreads, 0, s>>>(k, pool, slots, (IO*)state,
                                                                                        (IO*)y);
        return cudaGetLastError();
    });
}

}  // namespace layer
}  // namespace gdr
