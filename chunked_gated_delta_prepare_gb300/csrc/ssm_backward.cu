// The gradient of the selective state space scan (ssm.cuh has the forward's formulas), from its inputs alone.
//
// With g_t = dy_t silu(z_t), a_t = exp(Delta_t A) and dh_t the gradient of h_t:
//   dh_t = g_t C_t + a_{t+1} dh_{t+1}
//   dC_t[n] = sum_d g_t h_t          dB_t[n] = sum_d dh_t Delta_t x_t
//   r_t = sum_n dh_t B_t             w_t = dh_t a_t h_{t-1}           (the gradient of log a_t)
//   dx_t = r_t Delta_t + Dk g_t      dDelta_t = r_t x_t + sum_n A w_t    dA = sum_t Delta_t w_t
//   dz_t = dy_t (sum_n C_t h_t + Dk x_t) silu'(z_t)                   dDk = sum_t g_t x_t
//
// The reverse walk needs every h_t.  A first kernel scans forward and keeps the state before each chunk of 16 tokens (a
// quarter of a byte a token for every element of the state).  The main kernel takes the chunks of a segment from the last to
// the first; it forms the 8 states of half a chunk again, in registers, and walks back over them: 2.5 exponentials an
// element beside the first kernel's one, and no state passes through shared memory.  Segments as in the forward: the
// first kernel scans each from a zero state and in the same walk sums what its tokens send to the state before it (the
// decays multiplied up so far are all that takes); ssm_join joins both.
//
// Bound: issue slots, then fp32 operations, exponentials and shared memory, within a factor of two of each other.  A
// thread has 2 channels x 4 states.  Sums over n and over d cross threads: each thread leaves its terms of half a chunk
// in shared memory, in order of its number, and after the walk the block adds them, 16 bytes at a time; crossing lanes by
// shuffles token by token took twice the instructions.  dB and dC leave each block of channels as partial sums that a
// last kernel adds in order; dA, dDk and the bias likewise over the segments.  No atomics: the same bits in every run.
// Measured: 4 x 2048 tokens x 2048 channels x 16 states bf16 435 us for the main kernel (1.5 T exponentials/s) and 129 for
// the first one; 28 for the joins and sums.  The main kernel uses all 255 registers that two blocks an SM leave, and up to 32
// states keeps some 16 to 68 bytes a thread in local memory (252 for fp32 up to 8 states).
#include <algorithm>

#include "ssm.cuh"

namespace gdr {
namespace layer {
namespace {

constexpr int kThreads = 128;
constexpr int kChunk = 16, kHalf = 8;
constexpr int kDC = 2;                        // channels of a thread
constexpr int kMinSegment = 32;
constexpr int kLocalPerSm = 3, kMainPerSm = 2;   // blocks on an SM
constexpr float kLn2 = 0.6931471805599453f;

// Everything the kernels pass on: see plan().
struct Scratch {
    float *ckpt, *csum;           // [total / kChunk + segments][D][N], [...][D]
    float *ends, *dends, *sums;   // [segments][D][N] twice, [segments][D]
    float *part_bc;               // [blocks of a group][total][G][2][N]
    float *part_a, *part_d;       // [walks][D][N], [walks][2][D] (Dk, bias)
};

// Index of the checkpoint of the chunk that starts at token `row` of the axis, in segment `number`.
__device__ __forceinline__ int64_t ckpt_at(int64_t row, int64_t number) { return row / kChunk + number; }

// A block's tiles of T tokens x W channels in units of 8 channels, U of them a thread; the loads of a tile run ahead of
// its use.
template <typename IO, int T, int W> struct Units {
    static constexpr int V8 = W / 8, U = T * V8 <= kThreads ? 1 : T * V8 / kThreads, kStep = kThreads / V8;
    Raw8<IO> dt[U], x[U], dy[U], z[U];
    int col, tok;

    __device__ __forceinline__ Units() : col(threadIdx.x % V8 * 8), tok(threadIdx.x / V8) {}

    __device__ __forceinline__ void fetch(const Ssm& a, const IO* dyp, const Channels& ch, int64_t row, int live) {
        const int cc = ch.c0 + col;
        const bool vec8 = cc % (16 / (int)sizeof(IO)) == 0;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int k = tok + i * kStep, left = k < live ? ch.end - cc : 0;
            dt[i] = load8(reinterpret_cast<const IO*>(a.dt.p) + (row + k) * a.dt.ld + cc, left, a.dt.vec && vec8, cc);
            x[i] = load8(reinterpret_cast<const IO*>(a.x.p) + (row + k) * a.x.ld + cc, left, a.x.vec && vec8, cc);
            if (dyp) {
                dy[i] = load8(dyp + (row + k) * a.D + cc, left, a.vec && vec8, cc);
                if (a.z.p) z[i] = load8(reinterpret_cast<const IO*>(a.z.p) + (row + k) * a.z.ld + cc, left,
                                        a.z.vec && vec8, cc);
            }
        }
    }
    // Delta, Delta x and g (with_g) into shared memory [T][W]; zero past `live`, where nothing must happen.
    __device__ __forceinline__ void put(const Ssm& a, const float* bias, int live, bool with_g, float* s_delta,
                                        float* s_u, float* s_g) const {
        F2 d[U][4], u[U][4], g[U][4];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            pairs(dt[i], d[i]);
            pairs(x[i], u[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) d[i][j] = add2(d[i][j], reinterpret_cast<const F2*>(bias + col)[j]);
        }
        if (a.softplus)
#pragma unroll
            for (int i = 0; i < U; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) d[i][j] = softplus2(d[i][j]);
        if (with_g) {
#pragma unroll
            for (int i = 0; i < U; ++i) pairs(dy[i], g[i]);
            if (a.z.p)
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    F2 v[4];
                    pairs(z[i], v);
#pragma unroll
                    for (int j = 0; j < 4; ++j) g[i][j] = mul2(g[i][j], mul2(v[j], sigmoid2(v[j])));
                }
        }
        if (T * V8 < kThreads && tok >= T) return;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int k = tok + i * kStep, at = (k * W + col) / 2;
            const bool in = k < live;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                reinterpret_cast<F2*>(s_delta)[at + j] = in ? d[i][j] : 0;
                reinterpret_cast<F2*>(s_u)[at + j] = in ? mul2(u[i][j], d[i][j]) : 0;
                if (with_g) reinterpret_cast<F2*>(s_g)[at + j] = in ? g[i][j] : 0;
            }
        }
    }
};

// B (or C) of T tokens, NP states (zero past N and past `live`), likewise ahead of their use.
template <typename IO, int T, int NP> struct Values {
    static constexpr int M = (T * NP + kThreads - 1) / kThreads;
    IO v[M];

    __device__ __forceinline__ void fetch(const Ssm& a, const RowTensor& t, int group, int64_t row, int live) {
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const int k = (threadIdx.x + i * kThreads) / NP, m = (threadIdx.x + i * kThreads) % NP;
            v[i] = k < T && k < live && m < a.N
                       ? reinterpret_cast<const IO*>(t.p)[(row + k) * t.ld + group * a.N + m]
                       : from_f<IO>(0.f);
        }
    }
    __device__ __forceinline__ void put(float* s) const {
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const int at = threadIdx.x + i * kThreads;
            if (T * NP % kThreads == 0 || at < T * NP) s[at] = to_f(v[i]);
        }
    }
};

__device__ __forceinline__ void load_channels(const float* p, const Channels& ch, int width, float* s) {
    for (int i = threadIdx.x; i < width; i += kThreads) s[i] = p && ch.c0 + i < ch.end ? p[ch.c0 + i] : 0.f;
}

// Checkpoints of each segment from a zero state (the first segment of a sequence: from h0, so exact), what it leaves,
// its sum of Delta, and the gradient its own tokens send to the state before it.  2 channels x 8 states a thread.
template <typename IO, int LN>
__global__ void __launch_bounds__(kThreads, kLocalPerSm)
ssm_backward_local_kernel(Ssm a, const IO* __restrict__ dy, Scratch w) {
    constexpr int T = 8, W = kThreads / LN * kDC, NP = 8 * LN;
    __shared__ float4 s_delta[T * W / 4], s_u[T * W / 4], s_g[T * W / 4], s_b[T * NP / 4], s_c[T * NP / 4], s_bias[W / 4];
    const TileAt at = find_tile(a.q, blockIdx.x, a.seg);
    if (at.seq < 0) return;
    const bool last = (at.tile + 1) * a.seg >= at.len, back = at.tile > 0;
    const Channels ch = block_channels(a, W);
    const int q = threadIdx.x % LN, n = 8 * q, own = threadIdx.x / LN * kDC, c = ch.c0 + own;
    const int64_t state = (int64_t)a.D * a.N;
    const int64_t t0 = at.tile * a.seg, t1 = min(t0 + a.seg, at.len);

    Units<IO, T, W> in;
    Values<IO, T, NP> vb, vc;
    const auto fetch = [&](int64_t t) {
        const int live = (int)min((int64_t)T, t1 - t);
        in.fetch(a, back ? dy : nullptr, ch, at.start + t, live);
        vb.fetch(a, a.B, ch.group, at.start + t, live);
        if (back) vc.fetch(a, a.C, ch.group, at.start + t, live);
    };
    fetch(t0);
    load_channels(a.bias, ch, W, reinterpret_cast<float*>(s_bias));
    F2 A2[kDC][4], h[kDC][4], grown[kDC][4], dh[kDC][4];
    float sum[kDC];
    load_decay<kDC, 8>(a, c, ch.end, n, A2);
    load_states<kDC, 8>(back || !a.h0 ? nullptr : a.h0 + at.seq * state, a, c, ch.end, n, h);
#pragma unroll
    for (int i = 0; i < kDC; ++i) {
        sum[i] = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) grown[i][j] = both(1.f), dh[i][j] = 0;
    }
    __syncthreads();
    for (int64_t t = t0; t < t1; t += T) {
        const int live = (int)min((int64_t)T, t1 - t);
        if ((t - t0) % kChunk == 0) {
            const int64_t ck = ckpt_at(at.start + t, blockIdx.x);
            store_states<kDC, 8>(w.ckpt + ck * state, a, c, ch.end, n, h);
            if (back && q == 0)
#pragma unroll
                for (int i = 0; i < kDC; ++i)
                    if (c + i < ch.end) w.csum[ck * a.D + c + i] = sum[i];
            if (last && !back && t + kChunk >= t1) break;        // nobody asks for what the last chunk leaves
        }
        in.put(a, reinterpret_cast<const float*>(s_bias), live, back, reinterpret_cast<float*>(s_delta),
               reinterpret_cast<float*>(s_u), reinterpret_cast<float*>(s_g));
        vb.put(reinterpret_cast<float*>(s_b));
        if (back) vc.put(reinterpret_cast<float*>(s_c));
        __syncthreads();
        if (t + T < t1) fetch(t + T);
#pragma unroll 1
        for (int k = 0; k < live; ++k) {
            const float2 d = reinterpret_cast<const float2*>(s_delta)[(k * W + own) / 2];
            const float2 u = reinterpret_cast<const float2*>(s_u)[(k * W + own) / 2];
            const F2* pb = reinterpret_cast<const F2*>(s_b) + (k * NP + n) / 2;
            F2 b[4], cg[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = pb[j];
            if (back) {
                const float2 g = reinterpret_cast<const float2*>(s_g)[(k * W + own) / 2];
                const F2* pc = reinterpret_cast<const F2*>(s_c) + (k * NP + n) / 2;
#pragma unroll
                for (int j = 0; j < 4; ++j) cg[j] = pc[j];
#pragma unroll
                for (int i = 0; i < kDC; ++i) {
                    const F2 dd = both(i ? d.y : d.x), uu = both(i ? u.y : u.x), gg = both(i ? g.y : g.x);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const F2 e = decay2(A2[i][j], dd);
                        h[i][j] = fma2(e, h[i][j], mul2(uu, b[j]));
                        grown[i][j] = mul2(grown[i][j], e);
                        dh[i][j] = fma2(grown[i][j], mul2(gg, cg[j]), dh[i][j]);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < kDC; ++i) {
                    const F2 dd = both(i ? d.y : d.x), uu = both(i ? u.y : u.x);
#pragma unroll
                    for (int j = 0; j < 4; ++j) h[i][j] = fma2(decay2(A2[i][j], dd), h[i][j], mul2(uu, b[j]));
                }
            }
            sum[0] += d.x, sum[1] += d.y;
        }
        __syncthreads();
    }
    if (last && !back) return;                 // a sequence of one segment
    if (!last) store_states<kDC, 8>(w.ends + blockIdx.x * state, a, c, ch.end, n, h);
    if (back) store_states<kDC, 8>(w.dends + blockIdx.x * state, a, c, ch.end, n, dh);
    if (q == 0)
#pragma unroll
        for (int i = 0; i < kDC; ++i)
            if (c + i < ch.end) w.sums[(int64_t)blockIdx.x * a.D + c + i] = sum[i];
}

template <typename IO> struct Grads {
    const IO* dy;
    const float* dh_final;
    IO *dx, *ddt, *dz;
    float* dh0;
};

// The sum of LN neighbouring floats in shared memory.
template <int LN> __device__ __forceinline__ float lanes_total(const float* p) {
    if constexpr (LN == 2) {
        const float2 f = *reinterpret_cast<const float2*>(p);
        return f.x + f.y;
    } else {
        float s = 0.f;
#pragma unroll
        for (int m = 0; m < LN; m += 4) {
            const float4 f = *reinterpret_cast<const float4*>(p + m);
            s += (f.x + f.y) + (f.z + f.w);
        }
        return s;
    }
}

template <typename IO> __device__ __forceinline__ void store_pairs(IO* p, const F2 (&v)[4], int left, bool vec) {
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[2 * j] = unpack2(v[j]).x, f[2 * j + 1] = unpack2(v[j]).y;
    store_n(p, f, left, vec);
}

// Shared memory of the main kernel, in floats.  terms_bc: dB and dC terms [token of the half][B or C][thread], 4 states
// each; terms_n: r, y and sum A w, [token of the chunk][which][channel of the thread][thread].
// The terms of one token, value and channel parity: group g = thread / LN (2 channels) at term_at<LN>(g), so that the
// writers, and the readers of 4 neighbouring groups, both meet all banks.  With 2 lanes a channel (up to 8 states) the gap
// is 4 floats, where two writers share a bank: 8 would leave room for one block an SM, not the two that the registers and
// the walks' lengths count on (4 x 2048 x 2048 x 8 bf16 608 us, 421 so).
template <int LN> constexpr int kTermPad = LN == 2 ? 4 : 8;
template <int LN> constexpr int kTerms = 4 * (32 + kTermPad<LN>);
template <int LN> __device__ __forceinline__ int term_at(int g) { return g % 4 * (32 + kTermPad<LN>) + g / 4 * LN; }

template <int LN> struct MainTiles {
    static constexpr int W = kThreads / LN * kDC, NP = 4 * LN;
    static constexpr int delta = 0, u = delta + kChunk * W, g = u + kChunk * W, b = g + kChunk * W, c = b + kChunk * NP,
                         bias = c + kChunk * NP, D = bias + W, terms_bc = D + W,
                         terms_n = terms_bc + kHalf * 2 * kThreads * 4, total = terms_n + kChunk * 3 * kDC * kTerms<LN>;
    static_assert(terms_bc % 4 == 0 && terms_n % 4 == 0, "16-byte pieces");
    static_assert(kMainPerSm * (total * 4 + 1024) <= 228 * 1024, "the blocks fit an SM");
};

// span: segments (of the local kernel) of a block's walk.
template <typename IO, int LN>
__global__ void __launch_bounds__(kThreads, kMainPerSm) ssm_backward_kernel(Ssm a, int span, Grads<IO> o, Scratch w) {
    using S = MainTiles<LN>;
    constexpr int W = S::W, NP = S::NP;
    using In = Units<IO, kChunk, W>;
    extern __shared__ float4 smem4[];
    float* sm = reinterpret_cast<float*>(smem4);
    const int walk = a.seg * span;
    const TileAt at = find_tile(a.q, blockIdx.x, walk);
    const Channels ch = block_channels(a, W);
    const int q = threadIdx.x % LN, n = 4 * q, own = threadIdx.x / LN * kDC, c = ch.c0 + own;
    const int64_t state = (int64_t)a.D * a.N;

    In in;
    const int cc = ch.c0 + in.col, left = ch.end - cc;
    const bool vec8 = cc % (16 / (int)sizeof(IO)) == 0;
    F2 dA[kDC][2], dD[4], dbias[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) dA[0][j] = dA[1][j] = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) dD[j] = dbias[j] = 0;

    if (at.seq >= 0) {
        const int64_t t0 = at.tile * walk, t1 = min(t0 + walk, at.len);
        const int64_t first = first_tile(a.q, at.seq, a.seg);          // the sequence's first segment
        int64_t t = t1 > t0 ? t0 + (t1 - t0 - 1) / kChunk * kChunk : t0 - 1;
        Values<IO, kChunk, NP> vb, vc;
        F2 ckpt[kDC][2], start[kDC][2];                // the state before a chunk: its checkpoint, and in a later segment,
        float since[kDC];                              // whose checkpoints are local, the state before that decayed since
        const auto fetch = [&](int64_t from) {
            const int live = (int)min((int64_t)kChunk, t1 - from);
            const int64_t row = at.start + from, number = first + from / a.seg, ck = ckpt_at(row, number);
            load_states<kDC, 4>(w.ckpt + ck * state, a, c, ch.end, n, ckpt);
            if (from >= a.seg) {
                load_states<kDC, 4>(w.ends + number * state, a, c, ch.end, n, start);
#pragma unroll
                for (int i = 0; i < kDC; ++i) since[i] = c + i < ch.end ? w.csum[ck * a.D + c + i] : 0.f;
            }
            in.fetch(a, o.dy, ch, row, live);
            vb.fetch(a, a.B, ch.group, row, live);
            vc.fetch(a, a.C, ch.group, row, live);
        };
        if (t >= t0) fetch(t);
        load_channels(a.bias, ch, W, sm + S::bias);
        load_channels(a.Dk, ch, W, sm + S::D);
        F2 A2[kDC][2], dh[kDC][2];
        load_decay<kDC, 4>(a, c, ch.end, n, A2);
        const bool one = at.len <= a.seg;              // a sequence of one segment; else ssm_join has joined them
        const float* after = o.dh_final ? o.dh_final + at.seq * state : nullptr;
        if (!one) after = w.dends + (first + (t1 - 1) / a.seg) * state;
        load_states<kDC, 4>(after, a, c, ch.end, n, dh);
        __syncthreads();

        for (; t >= t0; t -= kChunk) {
            const int live = (int)min((int64_t)kChunk, t1 - t);
            const int64_t row = at.start + t;
            in.put(a, sm + S::bias, live, true, sm + S::delta, sm + S::u, sm + S::g);
            vb.put(sm + S::b);
            vc.put(sm + S::c);
            const In now = in;                         // what the elementwise end needs of this chunk
            F2 h0[kDC][2];
#pragma unroll
            for (int i = 0; i < kDC; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    h0[i][j] = t < a.seg ? ckpt[i][j]
                                         : fma2(decay2(A2[i][j], both(since[i])), start[i][j], ckpt[i][j]);
            __syncthreads();
            if (t > t0) fetch(t - kChunk);
            const float2* pd = reinterpret_cast<const float2*>(sm + S::delta + own);
            const float2* pu = reinterpret_cast<const float2*>(sm + S::u + own);
            const float2* pg = reinterpret_cast<const float2*>(sm + S::g + own);
            const F2* pb = reinterpret_cast<const F2*>(sm + S::b + n);
            const F2* pc = reinterpret_cast<const F2*>(sm + S::c + n);
#pragma unroll 1
            for (int half = live > kHalf ? 1 : 0; half >= 0; --half) {
                const int base = half * kHalf, tokens = min(kHalf, live - base);
                F2 hs[kHalf + 1][kDC][2];              // the states before each token of the half, and after the last
#pragma unroll
                for (int i = 0; i < kDC; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) hs[0][i][j] = h0[i][j];
                const auto step = [&](int k, const F2 (&from)[kDC][2], F2 (&to)[kDC][2]) {
                    const float2 d = pd[k * W / 2], u = pu[k * W / 2];
                    const F2 b[2] = {pb[k * NP / 2], pb[k * NP / 2 + 1]};
#pragma unroll
                    for (int i = 0; i < kDC; ++i) {
                        const F2 dd = both(i ? d.y : d.x), uu = both(i ? u.y : u.x);
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            to[i][j] = fma2(decay2(A2[i][j], dd), from[i][j], mul2(uu, b[j]));
                    }
                };
                if (half)
#pragma unroll 2
                    for (int k = 0; k < kHalf; ++k) step(k, hs[0], hs[0]);
#pragma unroll
                for (int k = 0; k < kHalf; ++k) step(base + k, hs[k], hs[k + 1]);
                if (half == 0 && live > kHalf) __syncthreads();        // the later half's dB and dC terms are used up
                F2 dAh[kDC][2];                        // dA of the half: short sums first keep its rounding small
#pragma unroll
                for (int i = 0; i < kDC; ++i) dAh[i][0] = dAh[i][1] = 0;
#pragma unroll
                for (int k = kHalf - 1; k >= 0; --k) {
                    const int tk = base + k;
                    const float2 d2 = pd[tk * W / 2], u2 = pu[tk * W / 2], g2 = pg[tk * W / 2];
                    const F2 b[2] = {pb[tk * NP / 2], pb[tk * NP / 2 + 1]}, cv[2] = {pc[tk * NP / 2], pc[tk * NP / 2 + 1]};
                    F2 dB[2], dC[2];
                    float* tn = sm + S::terms_n + tk * 3 * kDC * kTerms<LN> + term_at<LN>(threadIdx.x / LN) + q;
#pragma unroll
                    for (int i = 0; i < kDC; ++i) {
                        const F2 d = both(i ? d2.y : d2.x), u = both(i ? u2.y : u2.x), g = both(i ? g2.y : g2.x);
                        F2 y, r, s;                    // terms of C h, dh B and log2(e) A w
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const F2 e = decay2(A2[i][j], d);
                            dh[i][j] = fma2(g, cv[j], dh[i][j]);
                            y = j ? fma2(hs[k + 1][i][j], cv[j], y) : mul2(hs[k + 1][i][j], cv[j]);
                            r = j ? fma2(dh[i][j], b[j], r) : mul2(dh[i][j], b[j]);
                            dB[j] = i ? fma2(dh[i][j], u, dB[j]) : mul2(dh[i][j], u);
                            dC[j] = i ? fma2(hs[k + 1][i][j], g, dC[j]) : mul2(hs[k + 1][i][j], g);
                            dh[i][j] = mul2(e, dh[i][j]);
                            const F2 wt = mul2(dh[i][j], hs[k][i][j]);
                            s = j ? fma2(A2[i][j], wt, s) : mul2(A2[i][j], wt);
                            dAh[i][j] = fma2(d, wt, dAh[i][j]);
                        }
                        const float2 fr = unpack2(r), fy = unpack2(y), fs = unpack2(s);
                        tn[(0 * kDC + i) * kTerms<LN>] = fr.x + fr.y;
                        tn[(1 * kDC + i) * kTerms<LN>] = fy.x + fy.y;
                        tn[(2 * kDC + i) * kTerms<LN>] = fs.x + fs.y;
                    }
                    ulonglong2* tb = reinterpret_cast<ulonglong2*>(sm + S::terms_bc) + k * 2 * kThreads + threadIdx.x;
                    tb[0] = make_ulonglong2(dB[0], dB[1]);
                    tb[kThreads] = make_ulonglong2(dC[0], dC[1]);
                }
#pragma unroll
                for (int i = 0; i < kDC; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) dA[i][j] = add2(dA[i][j], dAh[i][j]);
                __syncthreads();

                // dB and dC of the half from this block's channels: 4 states of (token, B or C) an output, its terms
                // shared by `parts` neighbouring threads
                constexpr int outs = kHalf * 2 * LN, parts = outs < kThreads ? kThreads / outs : 1;
#pragma unroll
                for (int i = 0; i < (outs + kThreads - 1) / kThreads; ++i) {
                    const int out = (threadIdx.x + i * kThreads) / parts, part = threadIdx.x % parts;
                    const int qq = out % LN, bc = out / LN % 2, k = out / LN / 2;
                    const ulonglong2* p = reinterpret_cast<const ulonglong2*>(sm + S::terms_bc) + (k * 2 + bc) * kThreads + qq;
                    F2 lo = 0, hi = 0;
#pragma unroll
                    for (int j = 0; j < kThreads / LN / parts; ++j) {
                        const ulonglong2 f = p[(j * parts + part) * LN];
                        lo = add2(lo, f.x), hi = add2(hi, f.y);
                    }
                    const float2 f0 = unpack2(lo), f1 = unpack2(hi);
                    float v[4] = {f0.x, f0.y, f1.x, f1.y};
#pragma unroll
                    for (int m = 1; m < parts; m *= 2)
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[j] += __shfl_xor_sync(0xffffffffu, v[j], m);
                    if (part == 0 && k < tokens) {
                        const int m = 4 * qq;
                        float* to = w.part_bc +
                                    ((((int64_t)ch.block * a.q.total + row + base + k) * a.G + ch.group) * 2 + bc) * a.N + m;
                        if ((a.N & 3) == 0 && m < a.N) {
                            *reinterpret_cast<float4*>(to) = make_float4(v[0], v[1], v[2], v[3]);
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (m + j < a.N) to[j] = v[j];
                        }
                    }
                }
            }
            // the elementwise end: 8 channels of a token a unit, pairs of channels packed
#pragma unroll
            for (int i = 0; i < In::U; ++i) {
                const int k = in.tok + i * In::kStep;
                if (k >= live || left <= 0) continue;
                F2 v[3][4];                            // r, y, sum A w
#pragma unroll
                for (int j = 0; j < 3; ++j)
#pragma unroll
                    for (int x = 0; x < 8; x += 2) {   // channels x and x + 1 are one thread's two
                        const float* p = sm + S::terms_n + (k * 3 + j) * kDC * kTerms<LN> + term_at<LN>((in.col + x) / 2);
                        float f[2];
#pragma unroll
                        for (int m = 0; m < 2; ++m) f[m] = lanes_total<LN>(p + m * kTerms<LN>);
                        v[j][x / 2] = pack2(f[0], f[1]);
                    }
                const F2* delta = reinterpret_cast<const F2*>(sm + S::delta + k * W + in.col);
                const F2* g = reinterpret_cast<const F2*>(sm + S::g + k * W + in.col);
                const F2* D = reinterpret_cast<const F2*>(sm + S::D + in.col);
                const F2* bias = reinterpret_cast<const F2*>(sm + S::bias + in.col);
                F2 x[4], raw[4], out[4];
                pairs(now.x[i], x);
                pairs(now.dt[i], raw);
                const int64_t to = (row + k) * a.D + cc;
                if (a.z.p) {
                    F2 dy[4], z[4];
                    pairs(now.dy[i], dy);
                    pairs(now.z[i], z);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const F2 pre = a.Dk ? fma2(D[j], x[j], v[1][j]) : v[1][j];
                        out[j] = mul2(mul2(dy[j], pre), silu_slope2(z[j]));
                    }
                    store_pairs(o.dz + to, out, left, a.vec && vec8);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    out[j] = mul2(v[0][j], delta[j]);
                    if (a.Dk) out[j] = fma2(D[j], g[j], out[j]);
                }
                store_pairs(o.dx + to, out, left, a.vec && vec8);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    out[j] = fma2(v[0][j], x[j], mul2(both(kLn2), v[2][j]));
                    if (a.softplus) out[j] = mul2(out[j], sigmoid2(add2(raw[j], bias[j])));
                    dD[j] = fma2(g[j], x[j], dD[j]);
                    dbias[j] = add2(dbias[j], out[j]);
                }
                store_pairs(o.ddt + to, out, left, a.vec && vec8);
            }
            __syncthreads();
        }
        if (at.tile == 0 && o.dh0) store_states<kDC, 4>(o.dh0 + at.seq * state, a, c, ch.end, n, dh);
    }
    store_states<kDC, 4>(w.part_a + blockIdx.x * state, a, c, ch.end, n, dA);
    // dDk and the bias: over the threads that moved the same channels, in order
    ulonglong2* sums = reinterpret_cast<ulonglong2*>(sm + S::terms_bc);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        sums[2 * threadIdx.x + j] = make_ulonglong2(dD[2 * j], dD[2 * j + 1]);
        sums[2 * (kThreads + threadIdx.x) + j] = make_ulonglong2(dbias[2 * j], dbias[2 * j + 1]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * W; i += kThreads) {
        const int which = i / W, x = i % W;
        float v = 0.f;
        for (int m = 0; m < kThreads / In::V8; ++m)
            v += reinterpret_cast<const float*>(sums)[(which * kThreads + m * In::V8) * 8 + x];
        if (ch.c0 + x < ch.end) w.part_d[((int64_t)blockIdx.x * 2 + which) * a.D + ch.c0 + x] = v;
    }
}

// dB, dC [total][G][N] from the blocks' partial sums.
template <typename IO>
__global__ void __launch_bounds__(256) ssm_backward_bc_kernel(const float* __restrict__ part, int blocks, int64_t values,
                                                              int N, IO* __restrict__ dB, IO* __restrict__ dC) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < values; i += (int64_t)gridDim.x * 256) {
        float s = 0.f;
#pragma unroll 8
        for (int b = 0; b < blocks; ++b) s += part[b * values + i];
        const int64_t pair = i / N;                    // (token, group, B or C)
        (pair & 1 ? dC : dB)[pair / 2 * N + i % N] = from_f<IO>(s);
    }
}

int main_width(const SsmArgs& a) { return kThreads / ssm_lanes(a.N, 4) * kDC; }

int local_width(const SsmArgs& a) { return kThreads / ssm_lanes(a.N, 8) * kDC; }

// Tokens of a segment of the local kernel, and segments of a walk of the main one.
//
// Walks: a batch's sequences are cut where the waves of blocks times the tokens of a walk are least (kWalkStart tokens for
// a walk's start, about what a block takes before its first chunk); 7 walks of 293 tokens of a sequence measured 10 %
// less time than 2 of 1024 that left a sixth of the GPU idle.  Packed sequences, whose lengths the host does not know,
// have one wave, at least half of it for their tokens, the rest for the up to n walks that their ends add.  The local
// kernel's blocks are wider, so fewer: its segments are as many to a walk as fill its own wave.
constexpr int kWalkStart = 32, kMostCuts = 64;
struct Cuts {
    int seg, span;
};
Cuts cuts_of(const SsmArgs& a) {
    const int64_t blocks = ssm_blocks(a, main_width(a)), wave = kSms * kMainPerSm;
    const int64_t tokens = a.cu ? a.total : a.T, n = a.n;
    int64_t cuts = 1;
    if (a.cu) {
        const int64_t all = std::max<int64_t>(wave / blocks, 1);
        cuts = std::max(all - n, (all + 1) / 2);
    } else {
        const auto cost = [&](int64_t c) {
            return (n * c * blocks + wave - 1) / wave * ((tokens + c - 1) / c + kWalkStart);
        };
        for (int64_t c = 2; c <= kMostCuts && tokens / c >= kMinSegment; ++c)
            if (cost(c) < cost(cuts)) cuts = c;
    }
    const int64_t walk = std::max<int64_t>((tokens + cuts - 1) / cuts, kMinSegment);
    const int64_t walks = (a.cu ? 1 : n) * ((tokens + walk - 1) / walk);
    const int64_t wanted = kSms * kLocalPerSm / std::max<int64_t>(walks * ssm_blocks(a, local_width(a)), 1);
    const int64_t span = std::max<int64_t>(std::min(wanted, walk / kMinSegment), 1);
    const int64_t seg = ((walk + span - 1) / span + kChunk - 1) / kChunk * kChunk;
    return {(int)seg, (int)span};
}

size_t plan(const SsmArgs& a, float* base, Scratch* w) {
    const Seqs q{a.cu, a.total, a.T, (int)a.n};
    const Cuts cuts = cuts_of(a);
    const int64_t segments = tile_count(q, cuts.seg), walks = tile_count(q, cuts.seg * cuts.span);
    const int64_t ckpts = a.total / kChunk + segments;
    const int64_t D = a.D, DN = D * a.N, group_blocks = ssm_blocks(a, main_width(a)) / a.G;
    const bool split = a.cu || cuts.seg < a.T;
    size_t at = 0;
    const auto take = [&](int64_t floats) {
        float* p = base ? base + at : nullptr;
        at += (size_t)((floats + 63) / 64 * 64);       // 256-byte pieces
        return p;
    };
    w->ckpt = take(ckpts * DN);
    w->csum = take(split ? ckpts * D : 0);
    w->ends = take(split ? segments * DN : 0);
    w->dends = take(split ? segments * DN : 0);
    w->sums = take(split ? segments * D : 0);
    w->part_bc = take(group_blocks * a.total * a.G * 2 * a.N);
    w->part_a = take(walks * DN);
    w->part_d = take(walks * 2 * D);
    return at * sizeof(float);
}

}  // namespace

size_t ssm_backward_workspace(const SsmArgs& a) {
    Scratch w;
    return plan(a, nullptr, &w);
}

cudaError_t ssm_backward(const SsmArgs& a, const SsmTensors& t, const SsmGrads& g, float* workspace, cudaStream_t s) {
    Scratch w;
    plan(a, workspace, &w);
    Ssm k = ssm_of(a, t);
    const Cuts cuts = cuts_of(a);
    k.seg = cuts.seg;
    k.vec = (int64_t)a.D * (a.io == GDR_F32 ? 4 : 2) % 16 == 0;
    for (const void* p : {g.dy, (const void*)g.dx, (const void*)g.ddt, (const void*)g.dz})
        k.vec = k.vec && reinterpret_cast<uintptr_t>(p) % 16 == 0;
    const unsigned segments = (unsigned)tile_count(k.q, k.seg), walks = (unsigned)tile_count(k.q, k.seg * cuts.span);
    const bool split = a.cu || k.seg < a.T;
    cudaError_t e = ssm_types<8>(a.io, a.N, [&](auto io, auto lanes) {
        using IO = decltype(io);
        constexpr int LN = decltype(lanes)::value;
        ssm_backward_local_kernel<IO, LN>
            <<<dim3(segments, (unsigned)ssm_blocks(a, local_width(a))), kThreads, 0, s>>>(k, (const IO*)g.dy, w);
        return cudaGetLastError();
    });
    if (e == cudaSuccess && split) e = ssm_join(k, w.ends, w.dends, w.sums, g.dh_final, true, s);
    if (e != cudaSuccess) return e;
    e = ssm_types<4>(a.io, a.N, [&](auto io, auto lanes) {
        using IO = decltype(io);
        constexpr int LN = decltype(lanes)::value, bytes = MainTiles<LN>::total * 4;
        const Grads<IO> o{(const IO*)g.dy, g.dh_final, (IO*)g.dx, (IO*)g.ddt, (IO*)g.dz, g.dh0};
        if (cudaError_t x = cudaFuncSetAttribute(ssm_backward_kernel<IO, LN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 bytes))
            return x;
        ssm_backward_kernel<IO, LN>
            <<<dim3(walks, (unsigned)ssm_blocks(a, main_width(a))), kThreads, bytes, s>>>(k, cuts.span, o, w);
        if (cudaError_t x = cudaGetLastError()) return x;
        const int64_t values = a.total * a.G * 2 * a.N;
        if (values)
            ssm_backward_bc_kernel<IO><<<(unsigned)std::min<int64_t>((values + 255) / 256, kSms * 8), 256, 0, s>>>(
                w.part_bc, (int)(ssm_blocks(a, main_width(a)) / a.G), values, a.N, (IO*)g.dB, (IO*)g.dC);
        return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
    const int64_t D = a.D, DN = D * a.N;
    if (cudaError_t x = column_sum(w.part_a, walks, DN, DN, g.dA, 0, nullptr, s)) return x;
    if (!g.dDk && !g.dbias) return cudaSuccess;
    if (!g.dDk) return column_sum(w.part_d + D, walks, 2 * D, D, g.dbias, 0, nullptr, s);
    return column_sum(w.part_d, walks, 2 * D, D, g.dDk, g.dbias ? D : 0, g.dbias, s);
}

}  // namespace layer
}  // namespace gdr
