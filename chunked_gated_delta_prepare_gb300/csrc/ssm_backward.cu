// The gradient of the selective state space scan (ssm.cuh has the forward's formulas), from its inputs alone.
//
// With g_t = dy_t silu(z_t), a_t = exp(Delta_t A) and dh_t the gradient of h_t (sums over channels d of a group and
// states n written out):
//   dh_t = g_t C_t + a_{t+1} dh_{t+1}
//   dC_t[n] = sum_d g_t h_t          dB_t[n] = sum_d dh_t Delta_t x_t
//   r_t = sum_n dh_t B_t             w_t = dh_t a_t h_{t-1}           (the gradient of log a_t)
//   dx_t = r_t Delta_t + Dk g_t      dDelta_t = r_t x_t + sum_n A w_t    dA = sum_t Delta_t w_t
//   dz_t = dy_t (sum_n C_t h_t + Dk x_t) silu'(z_t)                   dDk = sum_t g_t x_t
//
// The reverse walk needs every h_t.  A first kernel scans forward and keeps the state before each chunk of 16 tokens (a
// quarter of a byte a token for every byte of state).  The main kernel takes the chunks of a segment from the last to
// the first; it forms the 8 states of half a chunk again, in registers, and walks back over them: 2.5 exponentials an
// element beside the first kernel's one, no state through shared memory.  Segments as in the forward: the first kernel
// scans each from a zero state and in the same walk sums what the gradient at the segment's start gets from its own
// tokens (the decays multiplied up so far are all that takes); the main kernel joins both over the other segments.
//
// Bound: fp32 operations (about 15 an element), then exponentials and shuffles.  A thread has 2 channels x 4 states:
// sums over n cross the channel's lanes, sums over d first the 2 channels, then the lanes that hold the same n, each
// value halved between the partners of a shuffle (12 shuffles a token for 8 elements).  dB and dC leave each block of
// channels as partial sums that a last kernel adds in order; dA, dDk and the bias likewise over the segments.  No
// atomics: the same bits in every run.
#include <algorithm>

#include "ssm.cuh"

namespace gdr {
namespace layer {
namespace {

constexpr int kChunk = 16, kHalf = 8;
constexpr int kDC = 2;                        // channels of a thread in the main kernel
constexpr int kMinSegment = 64;
constexpr int kWarps = kSsmThreads / 32;
constexpr float kLn2 = 0.6931471805599453f;

template <int LN> constexpr int local_channels() { return LN == 2 ? 2 : 4; }   // 4 would not fit 48 KB of tiles there

// Everything the kernels pass on: see plan().
struct Scratch {
    float *ckpt, *csum;           // [total / kChunk + segments][D][N], [...][D]
    float *ends, *dends, *sums;   // [segments][D][N] twice, [segments][D]
    float *part_bc;               // [blocks of a group][total][G][2][N]
    float *part_a, *part_d;       // [segments][D][N], [segments][2][D] (Dk, bias)
};

// Index of the checkpoint of the chunk that starts at token `row` of the axis, in segment `number`.
__device__ __forceinline__ int64_t ckpt_at(int64_t row, int64_t number) { return row / kChunk + number; }

// Delta, Delta x and g of a chunk's tokens into shared memory, [kChunk][W]; zero past `live` and past the channels.
template <typename IO, int W>
__device__ __forceinline__ void load_chunk(const Ssm& a, const IO* dy, const Channels& ch, int64_t row, int live,
                                           float4* s_delta, float4* s_u, float4* s_g) {
    for (int i = threadIdx.x; i < kChunk * W / 8; i += kSsmThreads) {
        const int k = i / (W / 8), col = i % (W / 8) * 8, cc = ch.c0 + col;
        const int left = k < live ? ch.end - cc : 0;
        float d[8], u[8], g[8], z[8];
        widen(load_row8<IO>(a.dt, row + k, cc, left), d);
        widen(load_row8<IO>(a.x, row + k, cc, left), u);
        if (dy) {
            widen(load8(dy + (row + k) * a.D + cc, left, a.vec && (cc & 7) == 0), g);
            if (a.z.p) widen(load_row8<IO>(a.z, row + k, cc, left), z);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            d[j] = j < left ? step_size(a, d[j], cc + j) : 0.f;
            u[j] = j < left ? u[j] * d[j] : 0.f;
            if (dy && a.z.p) g[j] = j < left ? g[j] * z[j] * sigmoid(z[j]) : 0.f;
        }
        const int at = (k * W + col) / 4;
        s_delta[at] = make_float4(d[0], d[1], d[2], d[3]), s_delta[at + 1] = make_float4(d[4], d[5], d[6], d[7]);
        s_u[at] = make_float4(u[0], u[1], u[2], u[3]), s_u[at + 1] = make_float4(u[4], u[5], u[6], u[7]);
        if (dy) s_g[at] = make_float4(g[0], g[1], g[2], g[3]), s_g[at + 1] = make_float4(g[4], g[5], g[6], g[7]);
    }
}

template <int P>
__device__ __forceinline__ void store_pairs(float* p, int c, int end, const F2 (&v)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const float2 f = unpack2(v[i]);
        if (c + 2 * i < end) p[2 * i] = f.x;
        if (c + 2 * i + 1 < end) p[2 * i + 1] = f.y;
    }
}

// Checkpoints of each segment from a zero state (the first segment of a sequence: from h0, so exact), what it leaves,
// its sum of Delta, and the gradient its own tokens send to the state before it.
template <typename IO, int LN>
__global__ void __launch_bounds__(kSsmThreads) ssm_backward_local_kernel(Ssm a, const IO* __restrict__ dy, Scratch w) {
    constexpr int DC = local_channels<LN>(), W = kSsmThreads / LN * DC, P = DC / 2;
    __shared__ float4 s_delta[kChunk * W / 4], s_u[kChunk * W / 4], s_g[kChunk * W / 4];
    __shared__ float2 s_b[kChunk * 4 * LN], s_c[kChunk * 4 * LN];
    const TileAt at = find_tile(a.q, blockIdx.x, a.seg);
    if (at.seq < 0) return;
    const bool last = (at.tile + 1) * a.seg >= at.len, back = at.tile > 0, split = back || !last;
    const Channels ch = block_channels(a, W);
    const int q = threadIdx.x % LN, n = 4 * q, own = threadIdx.x / LN * DC, c = ch.c0 + own;
    const int64_t state = (int64_t)a.D * a.N;

    F2 A2[4][P], h[4][P], grown[4][P], dh[4][P], sum[P];
    load_decay<DC>(a, c, ch.end, n, A2);
    load_states<DC>(back || !a.h0 ? nullptr : a.h0 + at.seq * state, a, c, ch.end, n, h);
#pragma unroll
    for (int i = 0; i < P; ++i) {
        sum[i] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) grown[j][i] = pack2(1.f, 1.f), dh[j][i] = 0;
    }
    const int64_t t0 = at.tile * a.seg, t1 = min(t0 + a.seg, at.len);
    for (int64_t t = t0; t < t1; t += kChunk) {
        const int live = (int)min((int64_t)kChunk, t1 - t);
        const int64_t row = at.start + t, ck = ckpt_at(row, blockIdx.x);
        store_states<DC>(w.ckpt + ck * state, a, c, ch.end, n, h);
        if (back && q == 0) store_pairs<P>(w.csum + ck * a.D + c, c, ch.end, sum);
        if (last && !back && t + kChunk >= t1) break;            // nobody asks for what the last chunk leaves
        load_chunk<IO, W>(a, back ? dy : nullptr, ch, row, live, s_delta, s_u, s_g);
        load_bc<IO, LN>(a, a.B, ch.group, row, live, kChunk, s_b);
        if (back) load_bc<IO, LN>(a, a.C, ch.group, row, live, kChunk, s_c);
        __syncthreads();
#pragma unroll 2
        for (int k = 0; k < live; ++k) {
            const F2* pd = reinterpret_cast<const F2*>(s_delta) + (k * W + own) / 2;
            const F2* pu = reinterpret_cast<const F2*>(s_u) + (k * W + own) / 2;
            const F2* pg = reinterpret_cast<const F2*>(s_g) + (k * W + own) / 2;
            const F2* pb = reinterpret_cast<const F2*>(s_b) + k * 4 * LN + n;
            const F2* pc = reinterpret_cast<const F2*>(s_c) + k * 4 * LN + n;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                sum[i] = add2(sum[i], pd[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const F2 e = ex2_2(mul2(A2[j][i], pd[i]));
                    h[j][i] = fma2(e, h[j][i], mul2(pu[i], pb[j]));
                    if (back) {
                        grown[j][i] = mul2(grown[j][i], e);
                        dh[j][i] = fma2(grown[j][i], mul2(pg[i], pc[j]), dh[j][i]);
                    }
                }
            }
        }
        __syncthreads();
    }
    if (!split) return;
    if (!last) store_states<DC>(w.ends + blockIdx.x * state, a, c, ch.end, n, h);
    if (back) store_states<DC>(w.dends + blockIdx.x * state, a, c, ch.end, n, dh);
    if (q == 0) store_pairs<P>(w.sums + (int64_t)blockIdx.x * a.D + c, c, ch.end, sum);
}

// Sums over the lanes that hold the same states (lane / LN differs) of v[0 .. 8), halving the values between partners
// while there are steps for it.  Lane group l is left with V values, the first of index first_value(l).
template <int LN> struct GroupSum {
    static constexpr int kGroups = 32 / LN;
    static constexpr int V = kGroups >= 8 ? 1 : 8 / kGroups;
    static __device__ __forceinline__ int first_value(int l) {
        int at = 0;
#pragma unroll
        for (int size = 4, bit = 1; size >= V; size /= 2, bit *= 2) at += l & bit ? size : 0;
        return at;
    }
    static __device__ __forceinline__ void sum(float (&v)[8], int l) {
        int mask = LN;
#pragma unroll
        for (int size = 4; size >= V; size /= 2, mask *= 2) {
            const bool up = l & (mask / LN);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i >= size) break;
                const float give = up ? v[i] : v[i + size], keep = up ? v[i + size] : v[i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, give, mask);
            }
        }
        if (kGroups == 16) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 16);
    }
};

template <typename IO> struct Grads {
    const IO* dy;
    const float* dh_final;
    IO *dx, *ddt, *dz;
    float* dh0;
};

template <typename IO, int LN>
__global__ void __launch_bounds__(kSsmThreads, 3) ssm_backward_kernel(Ssm a, Grads<IO> o, Scratch w) {
    constexpr int W = kSsmThreads / LN * kDC, V8 = W / 8;
    using Sum = GroupSum<LN>;
    __shared__ float4 s_delta[kChunk * W / 4], s_u[kChunk * W / 4], s_g[kChunk * W / 4];
    __shared__ float2 s_b[kChunk * 4 * LN], s_c[kChunk * 4 * LN];
    __shared__ float s_bc[kWarps][kHalf][8][LN];       // dB (values 0 .. 3 of each lane), dC (4 .. 7) of half a chunk
    const TileAt at = find_tile(a.q, blockIdx.x, a.seg);
    const Channels ch = block_channels(a, W);
    const int q = threadIdx.x % LN, n = 4 * q, own = threadIdx.x / LN * kDC, c = ch.c0 + own;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, group = lane / LN;
    const int64_t state = (int64_t)a.D * a.N;
    const int col8 = threadIdx.x % V8 * 8;             // the channels this thread moves to and from memory

    F2 A2[4][1], dh[4][1], dA[4][1];
    float dD[8], dbias[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) dA[j][0] = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) dD[j] = 0.f, dbias[j] = 0.f;

    if (at.seq >= 0) {
        load_decay<kDC>(a, c, ch.end, n, A2);
        load_states<kDC>(o.dh_final ? o.dh_final + at.seq * state : nullptr, a, c, ch.end, n, dh);
        const int64_t t0 = at.tile * a.seg, t1 = min(t0 + a.seg, at.len);
        const int64_t first = (int64_t)blockIdx.x - at.tile, segments = (at.len + a.seg - 1) / a.seg;
        // the decay of a whole segment on a state
        const auto through = [&](int64_t s, F2 (&v)[4][1], const float* add) {
            const float* p = w.sums + s * a.D + c;
            const F2 t = pack2(c < ch.end ? p[0] : 0.f, c + 1 < ch.end ? p[1] : 0.f);
            F2 e[4][1];
            load_states<kDC>(add + s * state, a, c, ch.end, n, e);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j][0] = fma2(ex2_2(mul2(A2[j][0], t)), v[j][0], e[j][0]);
        };
        for (int64_t s = first + segments - 1; s > (int64_t)blockIdx.x; --s) through(s, dh, w.dends);
        F2 start[4][1];                                // the state before a later segment, over its local checkpoints
        if (at.tile > 0) {
            load_states<kDC>(w.ends + first * state, a, c, ch.end, n, start);
            for (int64_t s = first + 1; s < (int64_t)blockIdx.x; ++s) through(s, start, w.ends);
        }

        for (int64_t t = t1 > t0 ? t0 + (t1 - t0 - 1) / kChunk * kChunk : t0 - 1; t >= t0; t -= kChunk) {
            const int live = (int)min((int64_t)kChunk, t1 - t);
            const int64_t row = at.start + t, ck = ckpt_at(row, blockIdx.x);
            F2 h0[4][1];
            load_states<kDC>(w.ckpt + ck * state, a, c, ch.end, n, h0);
            if (at.tile > 0) {
                const float* p = w.csum + ck * a.D + c;
                const F2 s = pack2(c < ch.end ? p[0] : 0.f, c + 1 < ch.end ? p[1] : 0.f);
#pragma unroll
                for (int j = 0; j < 4; ++j) h0[j][0] = fma2(ex2_2(mul2(A2[j][0], s)), start[j][0], h0[j][0]);
            }
            load_chunk<IO, W>(a, o.dy, ch, row, live, s_delta, s_u, s_g);
            load_bc<IO, LN>(a, a.B, ch.group, row, live, kChunk, s_b);
            load_bc<IO, LN>(a, a.C, ch.group, row, live, kChunk, s_c);
            __syncthreads();
            const F2* pd = reinterpret_cast<const F2*>(s_delta) + own / 2;
            const F2* pu = reinterpret_cast<const F2*>(s_u) + own / 2;
            const F2* pg = reinterpret_cast<const F2*>(s_g) + own / 2;
            const F2* pb = reinterpret_cast<const F2*>(s_b) + n;
            const F2* pc = reinterpret_cast<const F2*>(s_c) + n;
#pragma unroll 1
            for (int half = live > kHalf ? 1 : 0; half >= 0; --half) {
                F2 hs[kHalf + 1][4];                   // the states before each token of the half, and after the last
#pragma unroll
                for (int j = 0; j < 4; ++j) hs[0][j] = h0[j][0];
                if (half)
#pragma unroll 2
                    for (int k = 0; k < kHalf; ++k)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            hs[0][j] = fma2(ex2_2(mul2(A2[j][0], pd[k * W / 2])), hs[0][j],
                                            mul2(pu[k * W / 2], pb[k * 4 * LN + j]));
                const int base = half * kHalf;
#pragma unroll
                for (int k = 0; k < kHalf; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        hs[k + 1][j] = fma2(ex2_2(mul2(A2[j][0], pd[(base + k) * W / 2])), hs[k][j],
                                            mul2(pu[(base + k) * W / 2], pb[(base + k) * 4 * LN + j]));
#pragma unroll
                for (int k = kHalf - 1; k >= 0; --k) {
                    const int at_k = (base + k) * W / 2, bc_k = (base + k) * 4 * LN;
                    const F2 d = pd[at_k], u = pu[at_k], g = pg[at_k];
                    F2 y = 0, r = 0, s = 0;            // sums over n: C h, dh B, log2(e) A w
                    float v[8];                        // sums over d: dB, dC
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const F2 e = ex2_2(mul2(A2[j][0], d)), b = pb[bc_k + j], cc = pc[bc_k + j];
                        dh[j][0] = fma2(g, cc, dh[j][0]);
                        y = fma2(hs[k + 1][j], cc, y);
                        r = fma2(dh[j][0], b, r);
                        const float2 fb = unpack2(mul2(dh[j][0], u)), fc = unpack2(mul2(hs[k + 1][j], g));
                        v[j] = fb.x + fb.y;
                        v[4 + j] = fc.x + fc.y;
                        dh[j][0] = mul2(e, dh[j][0]);
                        const F2 wt = mul2(dh[j][0], hs[k][j]);
                        s = fma2(A2[j][0], wt, s);
                        dA[j][0] = fma2(d, wt, dA[j][0]);
                    }
                    // a channel's sums over its lanes: lane bit 0 keeps a channel, bit 1 splits (r, y) from s
                    const float2 fr = unpack2(r), fy = unpack2(y), fs = unpack2(s);
                    const bool odd = q & 1, two = q & 2;
                    float vr = (odd ? fr.y : fr.x) + __shfl_xor_sync(0xffffffffu, odd ? fr.x : fr.y, 1);
                    float vy = (odd ? fy.y : fy.x) + __shfl_xor_sync(0xffffffffu, odd ? fy.x : fy.y, 1);
                    float vs = (odd ? fs.y : fs.x) + __shfl_xor_sync(0xffffffffu, odd ? fs.x : fs.y, 1);
                    const int slot = (base + k) * W + own + odd;
                    if (LN == 2) {
                        reinterpret_cast<float*>(s_u)[slot] = vr;
                        reinterpret_cast<float*>(s_g)[slot] = vy;
                        reinterpret_cast<float*>(s_delta)[slot] = vs;
                    } else {
                        vr = (two ? vs : vr) + __shfl_xor_sync(0xffffffffu, two ? vr : vs, 2);
                        vy += __shfl_xor_sync(0xffffffffu, vy, 2);
#pragma unroll
                        for (int m = 4; m < LN; m *= 2) {
                            vr += __shfl_xor_sync(0xffffffffu, vr, m);
                            vy += __shfl_xor_sync(0xffffffffu, vy, m);
                        }
                        if (q < 2) {
                            reinterpret_cast<float*>(s_u)[slot] = vr;
                            reinterpret_cast<float*>(s_g)[slot] = vy;
                        } else if (q < 4) {
                            reinterpret_cast<float*>(s_delta)[slot] = vr;
                        }
                    }
                    Sum::sum(v, group);
                    if (Sum::kGroups < 16 || group < 8)
#pragma unroll
                        for (int i = 0; i < Sum::V; ++i) s_bc[warp][k][Sum::first_value(group) + i][q] = v[i];
                }
                __syncthreads();
                // dB and dC of the half from this block's channels: value (B or C, n) of token base + k
                const int tokens = min(kHalf, live - base);
                for (int i = threadIdx.x; i < tokens * 8 * LN; i += kSsmThreads) {
                    const int k = i / (8 * LN), bc = i / (4 * LN) % 2, m = i % (4 * LN);
                    if (m >= a.N) continue;
                    float t4 = 0.f;
#pragma unroll
                    for (int x = 0; x < kWarps; ++x) t4 += s_bc[x][k][bc * 4 + m % 4][m / 4];
                    const int blk = blockIdx.y - ch.group * ((a.per + W - 1) / W);
                    w.part_bc[((((int64_t)blk * a.q.total + row + base + k) * a.G + ch.group) * 2 + bc) * a.N + m] = t4;
                }
                __syncthreads();
            }
            for (int i = threadIdx.x; i < live * V8; i += kSsmThreads) {
                const int k = i / V8, cc = ch.c0 + col8, left = ch.end - cc;
                if (left <= 0) continue;
                const bool vec = a.vec && (cc & 7) == 0;
                const float* r = reinterpret_cast<const float*>(s_u) + k * W + col8;
                const float* y = reinterpret_cast<const float*>(s_g) + k * W + col8;
                const float* s = reinterpret_cast<const float*>(s_delta) + k * W + col8;
                float x[8], raw[8], g[8], z[8], out[8];
                widen(load_row8<IO>(a.x, row + k, cc, left), x);
                widen(load_row8<IO>(a.dt, row + k, cc, left), raw);
                widen(load8(o.dy + (row + k) * a.D + cc, left, vec), g);
                const int64_t to = (row + k) * a.D + cc;
                if (a.z.p) {
                    widen(load_row8<IO>(a.z, row + k, cc, left), z);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float sig = sigmoid(z[j]), Dx = a.Dk && j < left ? a.Dk[cc + j] * x[j] : 0.f;
                        out[j] = g[j] * (y[j] + Dx) * sig * fmaf(z[j], 1.f - sig, 1.f);
                        g[j] *= z[j] * sig;
                    }
                    store_n(o.dz + to, out, left, vec);
                }
                float ddt[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float v = raw[j] + (a.bias && j < left ? a.bias[cc + j] : 0.f);
                    const float delta = a.softplus ? softplus(v) : v;
                    out[j] = fmaf(r[j], delta, a.Dk && j < left ? a.Dk[cc + j] * g[j] : 0.f);
                    ddt[j] = fmaf(r[j], x[j], kLn2 * s[j]);
                    if (a.softplus) ddt[j] *= sigmoid(v);
                    if (j < left) {
                        dD[j] = fmaf(g[j], x[j], dD[j]);
                        dbias[j] += ddt[j];
                    }
                }
                store_n(o.dx + to, out, left, vec);
                store_n(o.ddt + to, ddt, left, vec);
            }
            __syncthreads();
        }
        if (at.tile == 0 && o.dh0) store_states<kDC>(o.dh0 + at.seq * state, a, c, ch.end, n, dh);
    }
    store_states<kDC>(w.part_a + blockIdx.x * state, a, c, ch.end, n, dA);
    // dDk and the bias: over the threads that moved the same channels, lanes first, then warps
    float (*sums)[V8][16] = reinterpret_cast<float (*)[V8][16]>(s_delta);
    static_assert(kWarps * V8 * 16 <= kChunk * W, "the sums fit the tile");
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int m = V8; m < 32; m *= 2) {
            dD[j] += __shfl_xor_sync(0xffffffffu, dD[j], m);
            dbias[j] += __shfl_xor_sync(0xffffffffu, dbias[j], m);
        }
        if (lane < V8) sums[warp][lane][j] = dD[j], sums[warp][lane][8 + j] = dbias[j];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < V8 * 16; i += kSsmThreads) {
        const int l = i / 16, j = i % 16, cc = ch.c0 + l * 8 + j % 8;
        float t = 0.f;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) t += sums[x][l][j];
        if (cc < ch.end) w.part_d[((int64_t)blockIdx.x * 2 + j / 8) * a.D + cc] = t;
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

int blocks_of_group(const SsmArgs& a) {
    const int width = kSsmThreads / ssm_lanes(a.N) * kDC;
    return (a.D / a.G + width - 1) / width;
}

// Tokens of a segment: two waves of blocks (3 an SM), or whole sequences where a batch has one wave of them.
int segment_of(const SsmArgs& a) {
    const int64_t blocks = (int64_t)a.G * blocks_of_group(a), wave = kSms * 3;
    int64_t seg;
    if (a.cu) seg = std::min(a.total, a.total * blocks / (2 * wave) + 1);
    else if (a.n * blocks >= wave) seg = a.T;
    else seg = (a.T + 2 * wave / (a.n * blocks) - 1) / (2 * wave / (a.n * blocks));
    seg = std::max<int64_t>(seg, kMinSegment);
    return (int)((seg + kChunk - 1) / kChunk * kChunk);
}

size_t plan(const SsmArgs& a, float* base, Scratch* w) {
    const Seqs q{a.cu, a.total, a.T, (int)a.n};
    const int64_t segments = tile_count(q, segment_of(a)), ckpts = a.total / kChunk + segments;
    const int64_t D = a.D, DN = D * a.N;
    const bool split = a.cu || segment_of(a) < a.T;
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
    w->part_bc = take((int64_t)blocks_of_group(a) * a.total * a.G * 2 * a.N);
    w->part_a = take(segments * DN);
    w->part_d = take(segments * 2 * D);
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
    k.seg = segment_of(a);
    k.vec = (int64_t)a.D * (a.io == GDR_F32 ? 4 : 2) % 16 == 0;
    for (const void* p : {g.dy, (const void*)g.dx, (const void*)g.ddt, (const void*)g.dz})
        k.vec = k.vec && reinterpret_cast<uintptr_t>(p) % 16 == 0;
    const int64_t segments = tile_count(k.q, k.seg);
    const cudaError_t e = ssm_types(a.io, a.N, [&](auto io, auto lanes) {
        using IO = decltype(io);
        constexpr int LN = decltype(lanes)::value, local = kSsmThreads / LN * local_channels<LN>();
        const Grads<IO> o{(const IO*)g.dy, g.dh_final, (IO*)g.dx, (IO*)g.ddt, (IO*)g.dz, g.dh0};
        const unsigned locals = (unsigned)(a.G * ((a.D / a.G + local - 1) / local));
        ssm_backward_local_kernel<IO, LN><<<dim3((unsigned)segments, locals), kSsmThreads, 0, s>>>(k, o.dy, w);
        if (cudaError_t x = cudaGetLastError()) return x;
        ssm_backward_kernel<IO, LN>
            <<<dim3((unsigned)segments, (unsigned)(a.G * blocks_of_group(a))), kSsmThreads, 0, s>>>(k, o, w);
        if (cudaError_t x = cudaGetLastError()) return x;
        const int64_t values = a.total * a.G * 2 * a.N;
        if (values)
            ssm_backward_bc_kernel<IO><<<(unsigned)std::min<int64_t>((values + 255) / 256, kSms * 8), 256, 0, s>>>(
                w.part_bc, blocks_of_group(a), values, a.N, (IO*)g.dB, (IO*)g.dC);
        return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
    if (cudaError_t x = column_sum(w.part_a, segments, (int64_t)a.D * a.N, (int64_t)a.D * a.N, g.dA, 0, nullptr, s))
        return x;
    if (g.dDk)
        if (cudaError_t x = column_sum(w.part_d, segments, 2 * (int64_t)a.D, a.D, g.dDk, 0, nullptr, s)) return x;
    if (g.dbias) return column_sum(w.part_d + a.D, segments, 2 * (int64_t)a.D, a.D, g.dbias, 0, nullptr, s);
    return cudaSuccess;
}

}  // namespace layer
}  // namespace gdr
