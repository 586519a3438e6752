// The short causal convolution of each channel over its own tokens, its gradient, and its single-token form.
//
//   p_t = b + sum_{j < W} w_j x_{t - W + 1 + j},   y_t = silu(p_t) or p_t;   x before the sequence: the W - 1 rows of
//   its state, or zero.  The state it leaves is the last W - 1 inputs.
//
// Bound: memory, x read once and y written once.  A thread takes 4 neighbouring channels down a run of tokens with the
// window of W inputs in registers, so each input is loaded once; only the W - 1 inputs before a run are read again.
// The next 12 tokens are on their way into the thread's own column of shared memory while these 4 are used: held in
// registers they cost occupancy (168 registers with 8 channels a thread, 92 with 4) and fewer were in flight.  Products
// go two channels at a time.  Measured: 16384 x 12288 bf16 in 11 packed sequences 134 us, 6.0 TB/s (0.90 of a copy's
// rate).  Rows that start anywhere (see Ring) are bound by instructions, three times as many a token: 310 us with 12287
// channels, fp32 8220 x 10838 155 us (0.69 of a copy's rate).
//
// Gradient: with dp_t = dy_t act'(p_t), p_t formed again from x,
//   dx_u = sum_j w_j dp_{u + W - 1 - j},  dw_j = sum_t dp_t x_{t - W + 1 + j},  db = sum_t dp_t.
// The same walk with a second window, of dp: at token t the gradient of x_{t - W + 1} is complete.  A run goes W - 1
// tokens past its end for the last of its dx.  dw and db are added in registers, then over the block's runs in shared
// memory, and leave as one row of partial sums a block, which column_sum adds in a fixed order.  Bound: issue slots and
// latency, 122 registers leaving 16 warps an SM.  Measured: 8192 x 6144 bf16 82 us, 3.7 TB/s, and 7 us for column_sum.
#include <algorithm>

#include "layer_common.cuh"
#include "layer_internal.h"

namespace gdr {
namespace layer {
namespace {

constexpr int kThreads = 128;
constexpr int N = 4, P = N / 2;      // channels of a thread, and pairs of them
constexpr int kRun = 64;             // tokens of a thread, fewer where there are few

// Lanes that share a token: the vectors of a row, at most 32 (a block's threads then hold kThreads / lanes runs).
int row_lanes(int64_t D) {
    int l = 1;
    while (l < 32 && l * N < D) l *= 2;
    return l;
}

struct Conv {
    Seqs q;
    int64_t D;
    RowTensor x;
    const void *w, *b, *state;
    int lanes, run;  // row_lanes; tokens of a thread
    bool silu;
    bool vec;        // rows of D elements on vectors' boundaries in every contiguous tensor (x.vec: in x)
    bool vec_w;      // w and b on 16-byte boundaries, which a thread's taps keep
};

// Input u of a sequence: a token (u >= 0), a row of its state, or zero.
template <typename IO>
__device__ __forceinline__ RawN<IO, N> input_at(const Conv& a, int seq, int64_t start, int64_t u, int64_t c, int back) {
    const int64_t left = a.D - c;
    if (u >= 0) return load_n<N>(reinterpret_cast<const IO*>(a.x.p) + (start + u) * a.x.ld + c, left, a.x.vec, c);
    if (a.state)
        return load_n<N>(reinterpret_cast<const IO*>(a.state) + ((int64_t)seq * back + back + u) * a.D + c, left, a.vec);
    return load_n<N>((const IO*)nullptr, 0, false);
}

// w[j]: tap j of the thread's channels, which lie side by side in memory
template <int W, typename IO>
__device__ __forceinline__ void load_taps(const Conv& a, int64_t c, F2 (&w)[W][P], F2 (&b)[P]) {
    IO e[N * W];
    const int64_t left = (a.D - c) * W;
#pragma unroll
    for (int i = 0; i < W; ++i)
        *reinterpret_cast<RawN<IO, N>*>(e + N * i) =
            load_n<N>(reinterpret_cast<const IO*>(a.w) + c * W + N * i, left - N * i, a.vec_w);
#pragma unroll
    for (int k = 0; k < P; ++k)
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][k] = pack2(to_f(e[2 * k * W + j]), to_f(e[(2 * k + 1) * W + j]));
    if (a.b) {
        pairs(load_n<N>(reinterpret_cast<const IO*>(a.b) + c, a.D - c, a.vec_w), b);
    } else {
#pragma unroll
        for (int k = 0; k < P; ++k) b[k] = 0;
    }
}

// Groups of kGroup tokens are used while kRing groups lie in, or are on their way into, the thread's own column of shared
// memory.  VEC: rows of aligned vectors, one copy each.  Other rows start anywhere; there a slot of 16 bytes takes the
// aligned words around a vector, and the neighbours' outputs are joined to aligned vectors.
constexpr int kGroup = 4;
template <typename IO, bool VEC> constexpr int kRing = VEC && sizeof(IO) == 2 ? 4 : VEC ? 2 : 3;
struct alignas(16) Words {
    uint32_t w[4];
};
template <typename IO, bool VEC> using Slot = std::conditional_t<VEC, RawN<IO, N>, Words>;
template <typename IO, bool VEC> using Ring = Slot<IO, VEC>[kRing<IO, VEC> * kGroup][kThreads];

// The thread's place in its row.
struct Place {
    int64_t c;            // first channel
    int left;             // channels from there on, 2 N at most
    int lane, lanes;      // lanes that share a token, neighbours of one warp
    unsigned mask;        // the lanes of them that have channels
    int live, last_left;  // their number, and `left` of the last one
    int before;           // the lane before, of the first one the last
};

// The tensor's first element where its address is an odd one's (fetch's base), else nullptr.
template <typename IO> __device__ __forceinline__ const IO* odd_start(const IO* p) {
    return sizeof(IO) == 2 && (reinterpret_cast<uintptr_t>(p) & 2) ? p : nullptr;
}

// p's elements [0, min(left, N)) on their way.  Without VEC by words: with a 16-bit type and an odd element first, the word
// around it brings the element before, which a tensor's first element does not have (base, where it is an odd one).
template <bool VEC, typename IO>
__device__ __forceinline__ void fetch(Slot<IO, VEC>* to, const IO* p, const Place& at, const IO* base) {
    if constexpr (VEC) {
        copy_ahead(to, p);
    } else if constexpr (sizeof(IO) == 4) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < at.left) copy_word(to->w + i, p + i, 4);
    } else {
        const int odd = (int)(reinterpret_cast<uintptr_t>(p) >> 1 & 1), have = 2 * (at.left + odd);
        const IO* q = p - odd;
        if (odd && base && p == base) reinterpret_cast<IO*>(to)[1] = p[0];
        else copy_word(to->w, q, min(have, 4));
        if (have > 4) copy_word(to->w + 1, q + 2, min(have - 4, 4));
        if (odd && have > 8) copy_word(to->w + 2, q + 4, min(have - 8, 4));
    }
}
template <bool VEC, typename IO>
__device__ __forceinline__ RawN<IO, N> take(const Slot<IO, VEC>& slot, const IO* p) {
    if constexpr (VEC) {
        return slot;
    } else {
        const Words s = slot;
        uint32_t w[5] = {s.w[0], s.w[1], s.w[2], s.w[3], 0};
        return shift_words<N, IO>(w, sizeof(IO) == 2 ? (int)(reinterpret_cast<uintptr_t>(p) & 2) : 0);
    }
}

// The thread's channels of a token to p.  Without VEC every lane of a token calls it at the same time, and takes from the
// lane before it what shares the aligned vector in which its own channels begin; the first lane stores the row's (or the
// block's) two ends.
template <bool VEC, typename IO>
__device__ __forceinline__ void store_token(IO* p, const F2 (&v)[P], const Place& at) {
    float f[N];
#pragma unroll
    for (int k = 0; k < P; ++k) f[2 * k] = unpack2(v[k]).x, f[2 * k + 1] = unpack2(v[k]).y;
    if constexpr (VEC) {
        store_n(p, f, N, true);
    } else {
        constexpr int block = N * (int)sizeof(IO), words = block / 4;
        RawN<IO, N> own;
#pragma unroll
        for (int i = 0; i < N; i += 2) from_f2(own.e + i, f[i], f[i + 1]);
        const int off = (int)(reinterpret_cast<uintptr_t>(p) % block), gone = off / (int)sizeof(IO);
        uint32_t w[2 * words + 1];
        w[2 * words] = 0;
#pragma unroll
        for (int i = 0; i < words; ++i) {
            w[words + i] = reinterpret_cast<const uint32_t*>(&own)[i];
            w[i] = __shfl_sync(at.mask, w[words + i], at.before, at.lanes);
        }
        // elements [-gone, N - gone) of p; the first lane's first ones are the last lane's last
        const RawN<IO, N> r = off ? shift_words<N, IO>(w, block - off) : own;
        IO* q = p - gone;
        const bool ends = gone > 0 && at.lane == 0;
        if (!ends && at.left >= N - gone) {
            store_raw(q, r, N, true);
        } else {
            const int tail = ends ? gone : 0, have = at.left + gone, end_have = at.last_left + gone - N;
            IO* e = q + at.live * N;
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i < (i < tail ? end_have : have)) (i < tail ? e : q)[i] = r.e[i];
        }
    }
}

// The run's outputs.  FAST: a whole run of aligned tokens.
template <typename IO, int W, bool SILU, bool VEC, bool FAST>
__device__ __forceinline__ void forward_run(const Conv& a, Ring<IO, VEC>& ring, const IO* xp, IO* yp, int run,
                                            const Place& at, F2 (&win)[W][P], const F2 (&w)[W][P], const F2 (&b)[P]) {
    constexpr int kBack = W - 1, S = kRing<IO, VEC>;
    const IO* base = odd_start(reinterpret_cast<const IO*>(a.x.p));
    const auto ahead = [&](int i0, int slot) {
        if (i0 < run)
#pragma unroll
            for (int i = 0; i < kGroup; ++i)
                if (FAST || i0 + i < run)
                    fetch<VEC>(&ring[slot * kGroup + i][threadIdx.x], xp + (i0 + i) * a.x.ld, at, base);
        copy_group();
    };
#pragma unroll
    for (int g = 0; g < S - 1; ++g) ahead(g * kGroup, g);
    for (int i0 = 0, slot = 0; i0 < run; i0 += kGroup, slot = slot + 1 == S ? 0 : slot + 1) {
        RawN<IO, N> raw[kGroup];
        ahead(i0 + (S - 1) * kGroup, slot == 0 ? S - 1 : slot - 1);
        copy_wait<S - 1>();
#pragma unroll
        for (int i = 0; i < kGroup; ++i)       // past the run's end: what the slot held
            raw[i] = take<VEC>(ring[slot * kGroup + i][threadIdx.x], xp + (i0 + i) * a.x.ld);
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
            pairs(raw[i], win[kBack]);
            F2 o[P];
#pragma unroll
            for (int k = 0; k < P; ++k) {
                o[k] = b[k];
#pragma unroll
                for (int j = 0; j < W; ++j) o[k] = fma2(w[j][k], win[j][k], o[k]);
#pragma unroll
                for (int j = 0; j < kBack; ++j) win[j][k] = win[j + 1][k];
                if (SILU) o[k] = silu2(o[k]);
            }
            if (FAST || i0 + i < run) store_token<VEC>(yp + (i0 + i) * a.D, o, at);
        }
    }
}

__device__ __forceinline__ Place place_of(const Conv& a) {
    Place p;
    p.lanes = a.lanes;
    p.lane = threadIdx.x % a.lanes;
    const int64_t first = (int64_t)blockIdx.y * a.lanes * N;
    const int here = (int)min((int64_t)a.lanes * N, a.D - first);
    p.c = first + p.lane * N;
    p.left = (int)max(min(a.D - p.c, (int64_t)2 * N), (int64_t)0);
    p.live = (here + N - 1) / N;
    p.last_left = (int)min(a.D - first - (p.live - 1) * N, (int64_t)2 * N);
    p.mask = (p.live == 32 ? ~0u : (1u << p.live) - 1) << (threadIdx.x % 32 - p.lane);
    p.before = p.lane == 0 ? p.live - 1 : p.lane - 1;
    return p;
}

template <typename IO, int W, bool SILU, bool VEC>
__global__ void __launch_bounds__(kThreads) conv_forward_kernel(Conv a, IO* __restrict__ y, IO* __restrict__ state_out) {
    constexpr int kBack = W - 1;
    __shared__ Ring<IO, VEC> ring;
    const Place place = place_of(a);
    const int sub = threadIdx.x / a.lanes, tile = a.run * (kThreads / a.lanes);
    const int64_t c = place.c;
    const int left = place.left;
    const TileAt at = find_tile(a.q, blockIdx.x, tile);
    const int64_t t0 = at.tile * tile + (int64_t)sub * a.run;
    if (at.seq < 0 || left <= 0 || (t0 >= at.len && t0 > 0)) return;

    F2 win[W][P], w[W][P], b[P];
    load_taps<W, IO>(a, c, w, b);
#pragma unroll
    for (int j = 0; j < kBack; ++j) pairs(input_at<IO>(a, at.seq, at.start, t0 - kBack + j, c, kBack), win[j]);

    const IO* xp = reinterpret_cast<const IO*>(a.x.p) + (at.start + t0) * a.x.ld + c;
    IO* yp = y + (at.start + t0) * a.D + c;
    const int run = (int)min((int64_t)a.run, at.len - t0);
    if (run == a.run) forward_run<IO, W, SILU, VEC, true>(a, ring, xp, yp, a.run, place, win, w, b);
    else forward_run<IO, W, SILU, VEC, false>(a, ring, xp, yp, run, place, win, w, b);
    if (t0 == 0 && state_out)                 // the first run leaves the state, an empty sequence's too
#pragma unroll
        for (int j = 0; j < kBack; ++j)
            store_raw(state_out + ((int64_t)at.seq * kBack + j) * a.D + c,
                      input_at<IO>(a, at.seq, at.start, at.len - kBack + j, c, kBack), left, a.vec);
}

// Where a run's gradients go, counted from its first token: token i gives dp_i and completes dx of i - (W - 1).
template <typename IO> struct BackwardRun {
    const IO *x, *dy, *dy_base;
    IO *dx, *d_state;             // d_state: the sequence's rows, one past the last
    const IO* d_state_out;        // the sequence's rows, shifted so that [u] is the one of input u
    int run, seen;                // tokens of the run; of them and the W - 1 after them those that exist
    int from, kept;               // first input with a gradient to store; first that is in the state the sequence left
};

// FAST: a whole run of aligned tokens inside a sequence, far from both its ends.
template <typename IO, int W, bool SILU, bool VEC, bool FAST>
__device__ __forceinline__ void backward_run(const Conv& a, Ring<IO, VEC> (&ring)[2], const BackwardRun<IO>& r,
                                             const Place& at, F2 (&win)[W][P], const F2 (&w)[W][P], const F2 (&b)[P],
                                             F2 (&dw)[W][P], F2 (&db)[P]) {
    constexpr int kBack = W - 1, S = kRing<IO, VEC>;
    const IO* base = odd_start(reinterpret_cast<const IO*>(a.x.p));
    F2 dp[W][P];
#pragma unroll
    for (int j = 0; j < kBack; ++j)
#pragma unroll
        for (int k = 0; k < P; ++k) dp[j][k] = 0;
    const auto ahead = [&](int i0, int slot) {
#pragma unroll
        for (int i = 0; i < kGroup; ++i)
            if (i0 + i < r.seen) {
                fetch<VEC>(&ring[0][slot * kGroup + i][threadIdx.x], r.x + (i0 + i) * a.x.ld, at, base);
                fetch<VEC>(&ring[1][slot * kGroup + i][threadIdx.x], r.dy + (i0 + i) * a.D, at, r.dy_base);
            }
        copy_group();
    };
    // token t: dp_t, and (OWN: a token of the run) its part of dw and db, then the gradient of input t - kBack
    const auto token = [&](int t, const RawN<IO, N>& x, const RawN<IO, N>& y, bool own) {
        const int u = t - kBack;
        F2 o[P];
        pairs(x, win[kBack]);
        pairs(y, dp[kBack]);
#pragma unroll
        for (int k = 0; k < P; ++k) {
            if (SILU) {
                F2 p = b[k];
#pragma unroll
                for (int j = 0; j < W; ++j) p = fma2(w[j][k], win[j][k], p);
                dp[kBack][k] = mul2(dp[kBack][k], silu_slope2(p));
            }
            if (!FAST && t >= r.seen) dp[kBack][k] = 0;    // not zero times an infinite input's slope
        }
        if (own)
#pragma unroll
            for (int k = 0; k < P; ++k) {
                db[k] = add2(db[k], dp[kBack][k]);
#pragma unroll
                for (int j = 0; j < W; ++j) dw[j][k] = fma2(dp[kBack][k], win[j][k], dw[j][k]);
            }
#pragma unroll
        for (int k = 0; k < P; ++k) {
            o[k] = mul2(w[0][k], dp[kBack][k]);
#pragma unroll
            for (int j = 1; j < W; ++j) o[k] = fma2(w[j][k], dp[kBack - j][k], o[k]);
#pragma unroll
            for (int j = 0; j < kBack; ++j) win[j][k] = win[j + 1][k], dp[j][k] = dp[j + 1][k];
        }
        if (u < r.from || (!FAST && u >= r.run)) return;
        if (!FAST && u >= r.kept) {                        // the gradient that comes through the state it left
            F2 e[P];
            pairs(load_n<N>(r.d_state_out + (int64_t)u * a.D, at.left, VEC), e);
#pragma unroll
            for (int k = 0; k < P; ++k) o[k] = add2(o[k], e[k]);
        }
        store_token<VEC>((FAST || u >= 0 ? r.dx : r.d_state) + (int64_t)u * a.D, o, at);
    };
    const auto taken = [&](int t, int slot, bool own) {
        token(t, take<VEC>(ring[0][slot][threadIdx.x], r.x + t * a.x.ld),
              take<VEC>(ring[1][slot][threadIdx.x], r.dy + t * a.D), own);
    };
#pragma unroll
    for (int g = 0; g < S - 1; ++g) ahead(g * kGroup, g);
    // past `seen` a slot gives what it held: no sum and no output has a part of it
    const int tokens = r.run + (FAST ? 0 : kBack);
    int slot = 0;
    for (int i0 = 0; i0 < tokens; i0 += kGroup, slot = slot + 1 == S ? 0 : slot + 1) {
        ahead(i0 + (S - 1) * kGroup, slot == 0 ? S - 1 : slot - 1);
        copy_wait<S - 1>();
#pragma unroll
        for (int i = 0; i < kGroup; ++i)
            if (FAST || i0 + i < tokens) taken(i0 + i, slot * kGroup + i, FAST || i0 + i < r.run);
    }
    if (FAST) {
        copy_wait<0>();
#pragma unroll
        for (int i = 0; i < kBack; ++i) taken(r.run + i, slot * kGroup + i, false);
    }
}

template <typename IO, int W, bool SILU, bool VEC>
__global__ void __launch_bounds__(kThreads)
conv_backward_kernel(Conv a, const IO* __restrict__ dy, const IO* __restrict__ d_state_out, IO* __restrict__ dx,
                     IO* __restrict__ d_state, float* __restrict__ partial) {
    constexpr int kBack = W - 1;
    __shared__ Ring<IO, VEC> ring[2];
    auto& sums = *reinterpret_cast<float(*)[kThreads][N * (W + 1) + 1]>(ring);   // after it; + 1: on different banks
    static_assert(sizeof(sums) <= sizeof(ring), "the sums fit");
    const Place place = place_of(a);
    const int sub = threadIdx.x / a.lanes, subs = kThreads / a.lanes, tile = a.run * subs;
    const int64_t c = place.c;
    const int left = place.left;
    const TileAt at = find_tile(a.q, blockIdx.x, tile);
    const int64_t t0 = at.tile * tile + (int64_t)sub * a.run;

    F2 dw[W][P], db[P];
#pragma unroll
    for (int k = 0; k < P; ++k) {
        db[k] = 0;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][k] = 0;
    }
    if (at.seq >= 0 && left > 0 && (t0 < at.len || t0 == 0)) {
        F2 win[W][P], w[W][P], b[P];
        load_taps<W, IO>(a, c, w, b);
#pragma unroll
        for (int j = 0; j < kBack; ++j) pairs(input_at<IO>(a, at.seq, at.start, t0 - kBack + j, c, kBack), win[j]);
        const int64_t row = at.start + t0, rows = (int64_t)at.seq * kBack;
        BackwardRun<IO> r;
        r.x = reinterpret_cast<const IO*>(a.x.p) + row * a.x.ld + c;
        r.dy = dy + row * a.D + c;
        r.dx = dx + row * a.D + c;
        r.d_state = d_state ? d_state + (rows + kBack) * a.D + c : nullptr;
        r.d_state_out = d_state_out ? d_state_out + (rows + kBack - (at.len - t0)) * a.D + c : nullptr;
        r.dy_base = odd_start(dy);
        r.run = (int)min((int64_t)a.run, at.len - t0);
        r.seen = (int)min((int64_t)r.run + kBack, at.len - t0);
        r.from = t0 == 0 && d_state ? -kBack : 0;
        r.kept = d_state_out ? (int)min(at.len - kBack - t0, (int64_t)r.run) : r.run;
        const bool inside = r.seen == a.run + kBack && r.from == 0 && r.kept == a.run;
        if (inside) backward_run<IO, W, SILU, VEC, true>(a, ring, r, place, win, w, b, dw, db);
        else backward_run<IO, W, SILU, VEC, false>(a, ring, r, place, win, w, b, dw, db);
    }
    copy_wait<0>();
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
#pragma unroll
        for (int j = 0; j < W; ++j)
            sums[threadIdx.x][k * W + j] = k & 1 ? unpack2(dw[j][k / 2]).y : unpack2(dw[j][k / 2]).x;
        sums[threadIdx.x][N * W + k] = k & 1 ? unpack2(db[k / 2]).y : unpack2(db[k / 2]).x;
    }
    __syncthreads();
    float* mine = partial + (int64_t)blockIdx.x * a.D * (W + 1);
    for (int i = threadIdx.x; i < a.lanes * N * (W + 1); i += kThreads) {
        const bool bias = i >= a.lanes * N * W;
        const int e = bias ? i - a.lanes * N * W : i, per = bias ? N : N * W;
        const int l = e / per, k = e % per;
        float s = 0.f;
        for (int m = 0; m < subs; ++m) s += sums[m * a.lanes + l][(bias ? N * W : 0) + k];
        const int64_t first = (int64_t)blockIdx.y * a.lanes * per + e;
        if (first < (bias ? a.D : a.D * W)) mine[(bias ? a.D * W : 0) + first] = s;
    }
}

// One token of a row: the state's W - 1 rows and the token are read at once, and the state goes back shifted.  Bound:
// latency (2.9 us for 64 x 6144 bf16, of which 6.4 MB at a copy's rate are 1.0).
template <typename IO, int W>
__global__ void __launch_bounds__(kThreads)
conv_step_kernel(Conv a, int64_t pool, const int* __restrict__ slots, IO* __restrict__ state, IO* __restrict__ y) {
    constexpr int kBack = W - 1;
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
    for (int j = 0; j < kBack; ++j) in[j] = load_own<N>(state + (slot * kBack + j) * a.D + c, left, a.vec);
    in[kBack] = load_n<N>(reinterpret_cast<const IO*>(a.x.p) + row * a.x.ld + c, left, a.x.vec, c);
    F2 w[W][P], b[P], v[P];
    load_taps<W, IO>(a, c, w, b);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        pairs(in[j], v);
#pragma unroll
        for (int k = 0; k < P; ++k) b[k] = fma2(w[j][k], v[k], b[k]);
    }
#pragma unroll
    for (int k = 0; k < P; ++k) {
        const float2 f = unpack2(a.silu ? silu2(b[k]) : b[k]);
        o[2 * k] = f.x, o[2 * k + 1] = f.y;
    }
    store_n(y + row * a.D + c, o, left, a.vec);
#pragma unroll
    for (int j = 0; j < kBack; ++j) store_raw(state + (slot * kBack + j) * a.D + c, in[j + 1], left, a.vec);
}

unsigned channel_blocks(int64_t D, int lanes) { return (unsigned)((D + lanes * N - 1) / (lanes * N)); }

// Tokens of a thread: kRun, halved down to 4 while the blocks are fewer than four an SM.  Taps and the window are loaded
// once a run, so long ones cost less (16384 x 12288: 144 us with 32, 134 with 64, 138 with 128; 8192 x 4096 30 and 28); at
// few tokens the blocks count for more (7252 x 1366: 22 us with 627 blocks of 32, 30 with 319 of 64).
int run_of(const ConvArgs& a) {
    const int lanes = row_lanes(a.D);
    const int64_t per = kThreads / lanes;
    int run = kRun;
    while (run > 4 && a.total / (run * per) * channel_blocks(a.D, lanes) < 4 * kSms) run /= 2;
    return run;
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
    const uintptr_t size = N * (a.io == GDR_F32 ? 4 : 2);
    k.vec = a.D % N == 0 && reinterpret_cast<uintptr_t>(state) % size == 0;
    for (const void* p : others) k.vec = k.vec && reinterpret_cast<uintptr_t>(p) % size == 0;
    k.x.vec = x.ld % N == 0 && reinterpret_cast<uintptr_t>(x.p) % size == 0;
    k.vec_w = reinterpret_cast<uintptr_t>(w) % 16 == 0 && reinterpret_cast<uintptr_t>(b) % 16 == 0;
    k.lanes = row_lanes(a.D);
    k.run = run_of(a);
    return k;
}

// Calls f with a value of the io type, the number of taps and whether the output goes through silu.
template <typename F> cudaError_t with_types(const ConvArgs& a, F f) {
    const auto act = [&](auto io, auto W) { return a.silu ? f(io, W, std::true_type()) : f(io, W, std::false_type()); };
    const auto taps = [&](auto io) {
        if (a.W == 2) return act(io, std::integral_constant<int, 2>());
        if (a.W == 3) return act(io, std::integral_constant<int, 3>());
        return act(io, std::integral_constant<int, 4>());
    };
    if (a.io == GDR_F32) return taps(float());
    if (a.io == GDR_BF16) return taps(__nv_bfloat16());
    return taps(__half());
}

}  // namespace

cudaError_t conv_forward(const ConvArgs& a, RowTensor x, const void* w, const void* b, const void* state, void* y,
                         void* state_out, cudaStream_t s) {
    const Conv k = conv_of(a, x, w, b, state, {y, state_out});
    const int64_t tiles = tile_count(k.q, k.run * (kThreads / k.lanes));
    return with_types(a, [&](auto io, auto taps, auto silu) {
        using IO = decltype(io);
        constexpr int W = decltype(taps)::value;
        constexpr bool kSilu = decltype(silu)::value;
        const auto kernel =
            k.vec && k.x.vec ? conv_forward_kernel<IO, W, kSilu, true> : conv_forward_kernel<IO, W, kSilu, false>;
        kernel<<<dim3((unsigned)tiles, channel_blocks(a.D, k.lanes)), kThreads, 0, s>>>(k, (IO*)y, (IO*)state_out);
        return cudaGetLastError();
    });
}

int64_t conv_partial_rows(const ConvArgs& a) {
    const Seqs q{a.cu, a.total, a.T, (int)a.n};
    return tile_count(q, run_of(a) * (kThreads / row_lanes(a.D)));
}

cudaError_t conv_backward(const ConvArgs& a, RowTensor x, const void* w, const void* b, const void* state,
                          const void* dy, const void* d_state_out, void* dx, float* dw, float* db, void* d_state,
                          float* partial, cudaStream_t s) {
    const Conv k = conv_of(a, x, w, b, state, {dy, d_state_out, dx, d_state});
    const int64_t tiles = conv_partial_rows(a);
    const cudaError_t e = with_types(a, [&](auto io, auto taps, auto silu) {
        using IO = decltype(io);
        constexpr int W = decltype(taps)::value;
        constexpr bool kSilu = decltype(silu)::value;
        const auto kernel =
            k.vec && k.x.vec ? conv_backward_kernel<IO, W, kSilu, true> : conv_backward_kernel<IO, W, kSilu, false>;
        kernel<<<dim3((unsigned)tiles, channel_blocks(a.D, k.lanes)), kThreads, 0, s>>>(
            k, (const IO*)dy, (const IO*)d_state_out, (IO*)dx, (IO*)d_state, partial);
        return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
    return column_sum(partial, tiles, a.D * (a.W + 1), a.D * a.W, dw, a.D, db, s);
}

cudaError_t conv_step(const ConvArgs& a, int64_t pool, const int* slots, RowTensor x, const void* w, const void* b,
                      void* state, void* y, cudaStream_t s) {
    const Conv k = conv_of(a, x, w, b, state, {y});
    return with_types(a, [&](auto io, auto taps, auto silu) {
        using IO = decltype(io);
        conv_step_kernel<IO, decltype(taps)::value>
            <<<dim3((unsigned)a.n, channel_blocks(a.D, kThreads)), kThreads, 0, s>>>(k, pool, slots, (IO*)state, (IO*)y);
        return cudaGetLastError();
    });
}

}  // namespace layer
}  // namespace gdr
