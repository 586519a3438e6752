// The gradient of the gated linear recurrence (formulas in lru.cuh).  With e_t the gradient of h_t:
//
//   e_t = dy_t + a_{t+1} e_{t+1}   (the last: + dh_final),   dh0 = a_1 e_1
//   dx = e s g,  di = e s x g (1 - g)
//   RATE:  dlog a = e a (h_{t-1} - g x a / s),  dr = -dlog a k q (1 - q),  dlam = -sum dlog a q c sigmoid(lam)
//   else:  dr = e a s (h_{t-1} - g x)
//
// Bound: memory.  One pass over the tiles from behind: as in the forward, with the gradient that reaches a tile from behind
// in the place of its state, which is the forward's kept one.
#include "lru.cuh"

namespace gdr {
namespace layer {
namespace {

constexpr int kBlocks = 2;   // an SM
template <typename IO> constexpr int kBuffers = sizeof(IO) == 2 ? 2 : 1;      // of tiles

template <typename IO, bool GATE> constexpr int lru_backward_smem() {
    return kBuffers<IO> * (GATE ? 4 : 3) * kLruTile * kLruCols * (int)sizeof(IO);
}

struct alignas(8) Run {      // of a run of tokens: its product of decays, its end from a zero state, and what it sends to the
    F2 decay, own, back;     // state before it with nothing behind it
};

// dlam: [tiles][D] partial sums, or nullptr.
template <typename IO, bool RATE, bool GATE>
__global__ void __launch_bounds__(kLruThreads, kBlocks)
lru_backward_kernel(Lru p, LruChain chain, LruRows dy, const float* __restrict__ kept, const float* __restrict__ dh_final,
                    IO* __restrict__ dx, IO* __restrict__ dr, IO* __restrict__ di, float* __restrict__ dlam,
                    float* __restrict__ dh0) {
    constexpr int B = kBuffers<IO>, N = kLruTile * kLruCols, IN = GATE ? 4 : 3;
    extern __shared__ uint4 smem[];
    __shared__ Run runs[kLruRuns][kLruPairs];
    __shared__ F2 sums[kLruRuns][kLruPairs];
    __shared__ F2 carry[kLruPairs];
    __shared__ LruPlan plans[3];
    IO* in = reinterpret_cast<IO*>(smem);                   // [B][IN][N]: r, x, dy, i

    if (threadIdx.x >= kLruWorkers) {                       // the guide
        lru_plan<true, RATE>(p, chain, 0, plans);
        lru_plan<true, RATE>(p, chain, 1, plans + 1);
        __syncthreads();
        const int pair = threadIdx.x % kLruPairs;
        for (unsigned turn = 0; plans[turn % 3].live; ++turn) {
            __syncthreads();                                // the tile is there
            lru_plan<true, RATE>(p, chain, turn + 2, plans + (turn + 2) % 3);
            const LruTile t = plans[turn % 3].t;
            const int ch = t.col * kLruCols + pair * 2, left = p.D - ch;
            const int64_t at = ((int64_t)t.number * p.cols + t.col) * kLruPairs + pair;
            const bool first = threadIdx.x < kLruWorkers + kLruPairs;  // the warp's other half does the same again
            F2 e = t.seq >= 0 ? state2(dh_final, (int64_t)t.seq * p.D + ch, left) : 0;
            __syncthreads();                                // the runs are there
            F2 d = both(1.f), b = both(0.f);
#pragma unroll
            for (int w = kLruRuns - 1; w >= 0; --w) {
                b = fma2(runs[w][pair].decay, b, runs[w][pair].back);
                d = mul2(runs[w][pair].decay, d);
            }
            if (t.seq >= 0) {
                if (first && t.to_tail && t.to_head) publish_map(chain.maps + at, d, b);
                if (t.to_tail) e = look_back<true>(chain, t, p.cols, pair, t.to_tail);
                const F2 end = fma2(d, e, b);
                if (first) {
                    if (t.to_head) publish_state(chain.states + at - (int64_t)p.cols * kLruPairs, end);
                    carry[pair] = e;
                    if (dh0 && !t.to_head) put_state2(dh0, (int64_t)t.seq * p.D + ch, end, left);
                }
            }
            __syncthreads();                                // the gradient from behind is there
            F2 slope = 0;
            if (RATE) slope = pack2(left > 0 ? rate_slope(p.lam[ch], p.c) : 0.f, left > 1 ? rate_slope(p.lam[ch + 1], p.c) : 0.f);
            __syncthreads();                                // the tile is done
            if (RATE) {                                     // the sums stay until the next tile's maps are there
                F2 sum = sums[0][pair];
#pragma unroll
                for (int w = 1; w < kLruRuns; ++w) sum = add2(sum, sums[w][pair]);
                if (first) put_state2(dlam, (int64_t)t.number * p.D + ch, mul2(sum, slope), left);
            }
        }
        return;
    }

    const int run = threadIdx.x / kLruPairs, pair = threadIdx.x % kLruPairs, row = run * kLruRun;
    const auto fetch = [&](unsigned turn) {
        if (plans[turn % 3].live) {
            const LruTile t = plans[turn % 3].t;
            IO* to = in + (turn % B) * IN * N;
            lru_fetch(p.r, t, p.D, to);
            lru_fetch(p.x, t, p.D, to + N);
            lru_fetch(dy, t, p.D, to + 2 * N);
            if (GATE) lru_fetch(p.i, t, p.D, to + 3 * N);
        }
        copy_group();
    };
    __syncthreads();
    fetch(0);
    if (B == 2) fetch(1);
    for (unsigned turn = 0; plans[turn % 3].live; ++turn) {
        const LruPlan& plan = plans[turn % 3];
        const int ch = plan.t.col * kLruCols + pair * 2, left = p.D - ch, len = plan.t.len;
        const bool some = plan.t.seq >= 0;
        F2 state = some ? state2(kept, (int64_t)plan.t.number * p.D + ch, left) : 0;
        copy_wait<B - 1>();
        __syncthreads();
        const F2 k = RATE ? *reinterpret_cast<const F2*>(plan.rates + pair * 2) : 0;
        const IO* from = in + (turn % B) * IN * N;
        F2 a[kLruRun], h[kLruRun], part[kLruRun], q[kLruRun], gate[kLruRun];
#pragma unroll
        for (int j = 0; j < kLruRun; ++j) {
            decay_and_part<RATE>(lru_read(from, row + j, pair), k, a[j], part[j], q[j]);
            h[j] = mul2(part[j], lru_read(from + N, row + j, pair));
            if (GATE) gate[j] = sigmoid2(lru_read(from + 3 * N, row + j, pair)), h[j] = mul2(h[j], gate[j]);
            if (row + j >= len) a[j] = both(1.f), h[j] = both(0.f);
        }
        Run m{both(1.f), both(0.f), both(0.f)};
#pragma unroll
        for (int j = 0; j < kLruRun; ++j) {
            m.own = fma2(a[j], m.own, h[j]);
            m.decay = mul2(m.decay, a[j]);
        }
#pragma unroll
        for (int j = kLruRun - 1; j >= 0; --j)
            if (row + j < len) m.back = mul2(a[j], add2(m.back, lru_read(from + 2 * N, row + j, pair)));
        runs[run][pair] = m;
        __syncthreads();
        for (int w = 0; w < run; ++w) state = fma2(runs[w][pair].decay, state, runs[w][pair].own);
#pragma unroll
        for (int j = 0; j < kLruRun; ++j) {
            const F2 after = fma2(a[j], state, h[j]);
            h[j] = state;                                   // the state in front of the token
            state = after;
        }
        F2 over = both(1.f), more = both(0.f);              // the map of the runs behind
        for (int w = kLruRuns - 1; w > run; --w) {
            more = fma2(runs[w][pair].decay, more, runs[w][pair].back);
            over = mul2(runs[w][pair].decay, over);
        }
        __syncthreads();
        F2 sum = both(0.f);
        if (some) {
            F2 e = fma2(over, carry[pair], more);
            const int64_t at = (plan.t.first + row) * p.D + ch;
#pragma unroll
            for (int j = kLruRun - 1; j >= 0; --j) {
                if (row + j >= len) continue;
                e = add2(e, lru_read(from + 2 * N, row + j, pair));
                const F2 x = lru_read(from + N, row + j, pair);
                const F2 eg = GATE ? mul2(e, gate[j]) : e, egx = mul2(eg, x), ea = mul2(e, a[j]);
                F2 dr_;
                if (RATE) {
                    // -dlog a q; 1 / s is finite where s = 0, and is multiplied by q or k = 0 there
                    const F2 ratio = mul2(a[j], rcp2_finite(part[j]));
                    const F2 base = mul2(q[j], fma2(mul2(egx, a[j]), ratio, neg2(mul2(ea, h[j]))));
                    sum = add2(sum, base);
                    dr_ = mul2(mul2(base, k), fma2(q[j], both(-1.f), both(1.f)));
                } else {
                    dr_ = mul2(mul2(a[j], part[j]), fma2(e, h[j], neg2(egx)));
                }
                const int64_t to = at + (int64_t)j * p.D;
                store2(dx + to, mul2(eg, part[j]), left, p.vec);
                store2(dr + to, dr_, left, p.vec);
                if (GATE) store2(di + to, mul2(mul2(egx, part[j]), fma2(gate[j], both(-1.f), both(1.f))), left, p.vec);
                e = ea;
            }
        }
        if (RATE) sums[run][pair] = sum;
        __syncthreads();
        fetch(turn + B);
    }
}

size_t up(size_t bytes) { return (bytes + 255) / 256 * 256; }

}  // namespace

// The chain, the partial sums of dlam, the kept states (where the call has none).
size_t lru_backward_workspace(const LruArgs& a, bool kept) {
    return up(lru_forward_workspace(a)) + (size_t)lru_tiles(a) * a.D * 4 * (kept ? 1 : 2);
}

cudaError_t lru_backward(const LruArgs& args, const LruTensors& t, const LruGrads& g, const float* kept, void* workspace,
                         cudaStream_t s) {
    float* partial = (float*)((char*)workspace + up(lru_forward_workspace(args)));
    if (!kept) {
        float* states = partial + lru_tiles(args) * args.D;
        if (cudaError_t e = lru_forward(args, t, nullptr, nullptr, states, workspace, s)) return e;
        kept = states;
    }
    const int64_t es = args.io == GDR_F32 ? 4 : 2;
    Lru p = lru_of(args, t);
    p.vec = true;
    for (const void* v : {(const void*)g.dx, (const void*)g.dr, (const void*)g.di}) p.vec = p.vec && lru_pairs(v, args.D, es);
    const LruRows dy = lru_rows(RowTensor{g.dy, args.D, reinterpret_cast<uintptr_t>(g.dy) % 16 == 0 && args.D * es % 16 == 0}, es);
    LruChain chain;
    if (cudaError_t e = lru_chain(args, workspace, &chain, s)) return e;
    const cudaError_t e = lru_types(args.io, t.lam, t.i.p, [&](auto io, auto rate, auto gate) {
        using IO = decltype(io);
        constexpr bool R = decltype(rate)::value, G = decltype(gate)::value;
        constexpr int bytes = lru_backward_smem<IO, G>();
        const auto kernel = lru_backward_kernel<IO, R, G>;
        if (cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) return err;
        kernel<<<std::min(p.tiles * p.cols, (unsigned)(kBlocks * kSms)), kLruThreads, bytes, s>>>(
            p, chain, dy, kept, g.dh_final, (IO*)g.dx, (IO*)g.dr, (IO*)g.di, partial, g.dh0);
        return cudaGetLastError();
    });
    if (e != cudaSuccess || !t.lam) return e;
    return column_sum(partial, lru_tiles(args), args.D, args.D, g.dlam, 0, nullptr, s);
}

}  // namespace layer
}  // namespace gdr
