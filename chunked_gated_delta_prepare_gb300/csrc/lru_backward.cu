// The gradient of the gated linear recurrence (formulas in lru.cuh).  With e_t the gradient of h_t:
//
//   e_t = dy_t + a_{t+1} e_{t+1}   (the last: + dh_final),   dh0 = a_1 e_1
//   dx = e s g,  di = e s x g (1 - g)
//   RATE:  dlog a = e a (h_{t-1} - g x a / s),  dr = -dlog a k q (1 - q),  dlam = -sum dlog a q c sigmoid(lam)
//   else:  dr = e a s (h_{t-1} - g x)
//
// Bound: memory.  Tiles as in the forward; the states in front of them are the forward's, the gradients behind them come
// from two kernels as the forward's states do, the first of which reads r and dy alone.
#include "lru.cuh"

namespace gdr {
namespace layer {

cudaError_t lru_states(const LruArgs& args, const LruTensors& t, float2* ends, float* kept, cudaStream_t s);

namespace {

struct alignas(8) Run {      // of a run of tokens: its product of decays, its end from a zero state, and what it sends back
    F2 decay, own, back;     // to the state before it with nothing behind it
};

// [tiles][D]: a tile's product of decays, and what it sends back.
template <typename IO, bool RATE>
__global__ void __launch_bounds__(kLruWarps * 32)
lru_back_ends_kernel(Lru p, const IO* __restrict__ dy, float2* __restrict__ ends) {
    __shared__ F2 run[kLruWarps][2][32];
    const LruTile t = lru_tile(p, blockIdx.x);
    if (t.seq < 0) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t0 = warp * kLruTokens;
    Rate k{0, 0};
    if (RATE) k = load_rate(p, t.ch, false);
    RawN<IO, 2> r[kLruTokens], g[kLruTokens];
    const int64_t row = t.first + t0;
#pragma unroll
    for (int j = 0; j < kLruTokens; ++j) {
        if (t0 + j >= t.len) continue;
        r[j] = load2((const IO*)p.r.p + (row + j) * p.r.ld + t.ch, t.left, p.r.vec);
        g[j] = load2(dy + (row + j) * p.D + t.ch, t.left, p.vec);
    }
    F2 decay = both(1.f), back = both(0.f);
#pragma unroll
    for (int j = kLruTokens - 1; j >= 0; --j) {
        if (t0 + j >= t.len) continue;
        const F2 a = decay_of<RATE>(wide2(r[j]), k);
        back = mul2(a, add2(back, wide2(g[j])));
        decay = mul2(decay, a);
    }
    run[warp][0][lane] = decay;
    run[warp][1][lane] = back;
    __syncthreads();
    if (warp) return;
#pragma unroll
    for (int w = kLruWarps - 2; w >= 0; --w) {
        if (w == kLruWarps - 2) decay = run[w + 1][0][lane], back = run[w + 1][1][lane];
        back = fma2(run[w][0][lane], back, run[w][1][lane]);
        decay = mul2(run[w][0][lane], decay);
    }
    const float2 d = unpack2(decay), b = unpack2(back);
    float2* out = ends + t.number * p.D + t.ch;
    if (t.left > 0) out[0] = make_float2(d.x, b.x);
    if (t.left > 1) out[1] = make_float2(d.y, b.y);
}

// behind [tiles][D]: what reaches the last state of a tile from behind it; dh0.
__global__ void __launch_bounds__(64)
lru_back_join_kernel(Lru p, const float2* __restrict__ ends, const float* __restrict__ dh_final, float* __restrict__ behind,
                     float* __restrict__ dh0) {
    const int ch = blockIdx.x * 64 + threadIdx.x;
    if (ch >= p.D) return;
    for (int s = blockIdx.y; s < p.q.n; s += gridDim.y) {
        int64_t start, len;
        seq_range(p.q, s, &start, &len);
        const int64_t first = first_tile(p.q, s, kLruTile), tiles = (len + kLruTile - 1) / kLruTile;
        float e = dh_final ? dh_final[(int64_t)s * p.D + ch] : 0.f;
#pragma unroll 8
        for (int64_t i = tiles - 1; i >= 0; --i) {
            const float2 b = ends[(first + i) * p.D + ch];
            behind[(first + i) * p.D + ch] = e;
            e = fmaf(b.x, e, b.y);
        }
        if (dh0) dh0[(int64_t)s * p.D + ch] = e;
    }
}

// dlam: [tiles][D] partial sums, or nullptr.
template <typename IO, bool RATE, bool GATE>
__global__ void __launch_bounds__(kLruWarps * 32)
lru_backward_kernel(Lru p, const IO* __restrict__ dy, const float* __restrict__ kept, const float* __restrict__ behind,
                    IO* __restrict__ dx, IO* __restrict__ dr, IO* __restrict__ di, float* __restrict__ dlam) {
    __shared__ Run run[kLruWarps][32];
    const LruTile t = lru_tile(p, blockIdx.x);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t0 = warp * kLruTokens;
    if (t.seq < 0 || t.len == 0) {
        if (RATE && warp == 0) put_state2(dlam, t.number * p.D + t.ch, both(0.f), t.left);
        return;
    }
    Rate k{0, 0};
    if (RATE) k = load_rate(p, t.ch, true);
    RawN<IO, 2> x[kLruTokens], r[kLruTokens], i[kLruTokens], g[kLruTokens];
    const int64_t row = t.first + t0;
#pragma unroll
    for (int j = 0; j < kLruTokens; ++j) {
        if (t0 + j >= t.len) continue;
        r[j] = load2((const IO*)p.r.p + (row + j) * p.r.ld + t.ch, t.left, p.r.vec);
        x[j] = load2((const IO*)p.x.p + (row + j) * p.x.ld + t.ch, t.left, p.x.vec);
        if (GATE) i[j] = load2((const IO*)p.i.p + (row + j) * p.i.ld + t.ch, t.left, p.i.vec);
        g[j] = load2(dy + (row + j) * p.D + t.ch, t.left, p.vec);
    }
    F2 a[kLruTokens], h[kLruTokens];          // h: the terms u, then the states in front of the tokens
    Run own{both(1.f), both(0.f), both(0.f)};
#pragma unroll
    for (int j = 0; j < kLruTokens; ++j) {
        a[j] = both(1.f), h[j] = both(0.f);
        if (t0 + j >= t.len) continue;
        F2 s;
        decay_and_part<RATE>(wide2(r[j]), k, a[j], s);
        h[j] = mul2(s, wide2(x[j]));
        if (GATE) h[j] = mul2(h[j], sigmoid2(wide2(i[j])));
        own.own = fma2(a[j], own.own, h[j]);
        own.decay = mul2(own.decay, a[j]);
    }
#pragma unroll
    for (int j = kLruTokens - 1; j >= 0; --j)
        if (t0 + j < t.len) own.back = mul2(a[j], add2(own.back, wide2(g[j])));
    run[warp][lane] = own;
    __syncthreads();
    F2 state = state2(kept, t.number * p.D + t.ch, t.left), e = state2(behind, t.number * p.D + t.ch, t.left);
    for (int w = 0; w < warp; ++w) state = fma2(run[w][lane].decay, state, run[w][lane].own);
    for (int w = kLruWarps - 1; w > warp; --w) e = fma2(run[w][lane].decay, e, run[w][lane].back);
#pragma unroll
    for (int j = 0; j < kLruTokens; ++j) {
        const F2 next = fma2(a[j], state, h[j]);
        h[j] = state;
        state = next;
    }
    F2 sum = both(0.f);
#pragma unroll
    for (int j = kLruTokens - 1; j >= 0; --j) {
        if (t0 + j >= t.len) continue;
        e = add2(e, wide2(g[j]));
        const F2 xv = wide2(x[j]);
        F2 gate = both(1.f), shut = both(0.f), q, rest, s, rs = 0, dr_;
        if (GATE) sigmoid_both2(wide2(i[j]), gate, shut);
        sigmoid_both2(wide2(r[j]), q, rest);
        const F2 eg = mul2(e, gate), egx = mul2(eg, xv);
        if (RATE) {
            const F2 kq = mul2(k.k, q), m = one_less(mul2(kq, both(-2.f)), a[j]);
            rs = rsqrt2(m);
            s = mul2(m, rs);
            // dlog a = keep - part / s; 1 / s is finite where s = 0, and meets q (k, its slope) first, which are 0 there
            const F2 keep = mul2(mul2(e, a[j]), h[j]), part = mul2(mul2(egx, a[j]), a[j]);
            dr_ = mul2(rest, fma2(part, mul2(kq, rs), neg2(mul2(keep, kq))));
            const F2 lq = mul2(k.slope, q);
            sum = add2(sum, fma2(part, mul2(lq, rs), neg2(mul2(keep, lq))));
        } else {
            s = rest;
            dr_ = mul2(mul2(a[j], s), fma2(e, h[j], neg2(egx)));
        }
        const int64_t at = (row + j) * p.D + t.ch;
        store2(dx + at, mul2(eg, s), t.left, p.vec);
        store2(dr + at, dr_, t.left, p.vec);
        if (GATE) store2(di + at, mul2(mul2(egx, s), shut), t.left, p.vec);
        e = mul2(a[j], e);
    }
    if (!RATE) return;
    __syncthreads();                          // the runs have been read
    F2* sums = reinterpret_cast<F2*>(&run[0][0]);
    sums[warp * 32 + lane] = sum;
    __syncthreads();
    if (warp) return;
#pragma unroll
    for (int w = 1; w < kLruWarps; ++w) sum = add2(sum, sums[w * 32 + lane]);
    put_state2(dlam, t.number * p.D + t.ch, sum, t.left);
}

}  // namespace

// The forward's part (without kept), the tiles' ends, the gradients behind the tiles, the partial sums of dlam.
size_t lru_backward_workspace(const LruArgs& a, bool kept) {
    return (size_t)lru_tiles(a) * a.D * 4 * (kept ? 4 : 5);
}

cudaError_t lru_backward(const LruArgs& args, const LruTensors& t, const LruGrads& g, const float* kept, float* workspace,
                         cudaStream_t s) {
    const int64_t cells = lru_tiles(args) * args.D;
    float2* ends = (float2*)workspace;
    float *behind = workspace + 2 * cells, *rest = behind + cells;
    if (!kept) {
        if (cudaError_t e = lru_states(args, t, ends, rest, s)) return e;
        kept = rest;
        rest += cells;
    }
    Lru p = lru_of(args, t);
    p.vec = true;
    for (const void* v : {g.dy, (const void*)g.dx, (const void*)g.dr, (const void*)g.di})
        p.vec = p.vec && lru_pairs(v, args.D, args.io == GDR_F32 ? 4 : 2);
    const unsigned blocks = (unsigned)(lru_tiles(args) * p.cols);
    const cudaError_t e = lru_types(args.io, t.lam, t.i.p, [&](auto io, auto rate, auto gate) {
        using IO = decltype(io);
        constexpr bool R = decltype(rate)::value, G = decltype(gate)::value;
        lru_back_ends_kernel<IO, R><<<blocks, kLruWarps * 32, 0, s>>>(p, (const IO*)g.dy, ends);
        if (cudaError_t err = cudaGetLastError()) return err;
        const dim3 grid((unsigned)((args.D + 63) / 64), (unsigned)std::min<int64_t>(args.n, 65535));
        lru_back_join_kernel<<<grid, 64, 0, s>>>(p, ends, g.dh_final, behind, g.dh0);
        if (cudaError_t err = cudaGetLastError()) return err;
        lru_backward_kernel<IO, R, G><<<blocks, kLruWarps * 32, 0, s>>>(p, (const IO*)g.dy, kept, behind, (IO*)g.dx,
                                                                        (IO*)g.dr, (IO*)g.di, rest);
        return cudaGetLastError();
    });
    if (e != cudaSuccess || !t.lam) return e;
    return column_sum(rest, lru_tiles(args), args.D, args.D, g.dlam, 0, nullptr, s);
}

}  // namespace layer
}  // namespace gdr
