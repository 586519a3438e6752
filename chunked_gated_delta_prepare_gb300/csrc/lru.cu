// The gated linear recurrence over prompts and batches, and its single-token step (formulas in lru.cuh).
//
// Bound: memory.  One pass: a tile's rows arrive in shared memory while the block works on the tile before, a thread forms
// the decays a and terms u of its run of 8 tokens in registers, the runs' maps h -> h * decay + own are joined through
// shared memory, the tile's state comes from the tiles before it (look_back), and the run is gone over again from its state.
#include "lru.cuh"

namespace gdr {
namespace layer {
namespace {

struct alignas(16) Map {     // what a run of tokens makes of state h: h * decay + own
    F2 decay, own;
};

constexpr int kBlocks = 3;   // an SM
template <typename IO> constexpr int kBuffers = sizeof(IO) == 2 ? 2 : 1;      // of tiles

template <typename IO, bool GATE> constexpr int lru_forward_smem() {
    return kBuffers<IO> * (GATE ? 3 : 2) * kLruTile * kLruCols * (int)sizeof(IO);
}

// y, kept and h_final may each be nullptr.
template <typename IO, bool RATE, bool GATE>
__global__ void __launch_bounds__(kLruThreads, kBlocks)
lru_forward_kernel(Lru p, LruChain chain, IO* __restrict__ y, float* __restrict__ kept, float* __restrict__ h_final) {
    constexpr int B = kBuffers<IO>, N = kLruTile * kLruCols, IN = GATE ? 3 : 2;
    extern __shared__ uint4 smem[];
    __shared__ Map runs[kLruRuns][kLruPairs];
    __shared__ F2 carry[kLruPairs];
    __shared__ LruPlan plans[3];
    IO* in = reinterpret_cast<IO*>(smem);                   // [B][IN][N]: r, x, i

    if (threadIdx.x >= kLruWorkers) {                       // the guide
        lru_plan<false, RATE>(p, chain, 0, plans);
        lru_plan<false, RATE>(p, chain, 1, plans + 1);
        __syncthreads();
        const int pair = threadIdx.x % kLruPairs;
        for (unsigned turn = 0; plans[turn % 3].live; ++turn) {
            __syncthreads();                                // the tile is there
            lru_plan<false, RATE>(p, chain, turn + 2, plans + (turn + 2) % 3);
            const LruTile t = plans[turn % 3].t;
            const int ch = t.col * kLruCols + pair * 2, left = p.D - ch;
            const int64_t at = ((int64_t)t.number * p.cols + t.col) * kLruPairs + pair;
            const bool first = threadIdx.x < kLruWorkers + kLruPairs;  // the warp's other half does the same again
            F2 state = t.seq >= 0 ? state2(p.h0, (int64_t)t.seq * p.D + ch, left) : 0;
            __syncthreads();                                // the runs' maps are there
            Map all = runs[0][pair];
#pragma unroll
            for (int w = 1; w < kLruRuns; ++w) {
                const Map n = runs[w][pair];
                all.own = fma2(n.decay, all.own, n.own);
                all.decay = mul2(n.decay, all.decay);
            }
            if (t.seq >= 0) {
                if (first && t.to_tail && t.to_head) publish_map(chain.maps + at, all.decay, all.own);
                if (t.to_head) state = look_back<false>(chain, t, p.cols, pair, t.to_head);
                const F2 end = fma2(all.decay, state, all.own);
                if (first) {
                    if (t.to_tail) publish_state(chain.states + at + (int64_t)p.cols * kLruPairs, end);
                    carry[pair] = state;
                    if (kept) put_state2(kept, (int64_t)t.number * p.D + ch, state, left);
                    if (h_final && !t.to_tail) put_state2(h_final, (int64_t)t.seq * p.D + ch, end, left);
                }
            }
            __syncthreads();                                // the state is there
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
            if (GATE) lru_fetch(p.i, t, p.D, to + 2 * N);
        }
        copy_group();
    };
    __syncthreads();
    fetch(0);
    if (B == 2) fetch(1);
    for (unsigned turn = 0; plans[turn % 3].live; ++turn) {
        copy_wait<B - 1>();
        __syncthreads();
        const LruPlan& plan = plans[turn % 3];
        F2 a[kLruRun], u[kLruRun];
        {
            const F2 k = RATE ? *reinterpret_cast<const F2*>(plan.rates + pair * 2) : 0;
            const IO* from = in + (turn % B) * IN * N;
#pragma unroll
            for (int j = 0; j < kLruRun; ++j) {
                F2 s, q;
                decay_and_part<RATE>(lru_read(from, row + j, pair), k, a[j], s, q);
                u[j] = mul2(s, lru_read(from + N, row + j, pair));
                if (GATE) u[j] = mul2(u[j], sigmoid2(lru_read(from + 2 * N, row + j, pair)));
            }
        }
        const int len = plan.t.len;
        if (len < kLruTile)
#pragma unroll
            for (int j = 0; j < kLruRun; ++j)
                if (row + j >= len) a[j] = both(1.f), u[j] = both(0.f);
        Map m{a[0], u[0]};
#pragma unroll
        for (int j = 1; j < kLruRun; ++j) {
            m.own = fma2(a[j], m.own, u[j]);
            m.decay = mul2(a[j], m.decay);
        }
        runs[run][pair] = m;
        __syncthreads();
        fetch(turn + B);
        m = Map{both(1.f), both(0.f)};                      // of the runs in front of the thread's
        for (int w = 0; w < run; ++w) {
            const Map n = runs[w][pair];
            m.own = fma2(n.decay, m.own, n.own);
            m.decay = mul2(n.decay, m.decay);
        }
        __syncthreads();
        if (y && plan.t.seq >= 0) {
            F2 h = fma2(m.decay, carry[pair], m.own);
            const int ch = plan.t.col * kLruCols + pair * 2, left = p.D - ch;
            IO* yp = y + (plan.t.first + row) * p.D + ch;
#pragma unroll
            for (int j = 0; j < kLruRun; ++j) {
                h = fma2(a[j], h, u[j]);
                if (row + j < len) store2(yp, h, left, p.vec);
                yp += p.D;
            }
        }
    }
}

template <typename IO, bool RATE, bool GATE>
__global__ void __launch_bounds__(128)
lru_step_kernel(Lru p, int64_t rows, int64_t pool, const int* __restrict__ slots, float* __restrict__ h, IO* __restrict__ y) {
    const int ch = (blockIdx.x * 128 + threadIdx.x) * 2, left = p.D - ch;
    if (left <= 0) return;
    const auto in_pairs = [](const LruRows& v) { return v.unit >= (sizeof(IO) == 2 ? 4 : 16); };
    F2 k = 0;
    if (RATE) k = pack2(rate_of(p.lam[ch], p.c), left > 1 ? rate_of(p.lam[ch + 1], p.c) : 0.f);
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        const int64_t slot = slots ? slots[row] : row;
        IO* yp = y + row * p.D + ch;
        if (slot < 0 || slot >= pool) {
            store2(yp, both(0.f), left, p.vec);
            continue;
        }
        F2 a, s, q;
        decay_and_part<RATE>(wide2(load2((const IO*)p.r.p + row * p.r.ld + ch, left, in_pairs(p.r))), k, a, s, q);
        F2 u = mul2(s, wide2(load2((const IO*)p.x.p + row * p.x.ld + ch, left, in_pairs(p.x))));
        if (GATE) u = mul2(u, sigmoid2(wide2(load2((const IO*)p.i.p + row * p.i.ld + ch, left, in_pairs(p.i)))));
        const F2 n = fma2(a, state2(h, slot * p.D + ch, left), u);
        put_state2(h, slot * p.D + ch, n, left);
        store2(yp, n, left, p.vec);
    }
}

}  // namespace

int64_t lru_tiles(const LruArgs& a) { return tile_count(Seqs{a.cu, a.total, a.T, (int)a.n}, kLruTile); }

size_t lru_forward_workspace(const LruArgs& a) {
    return lru_one_tile_each(a) ? 0 : lru_chain_bytes(lru_tiles(a), (a.D + kLruCols - 1) / kLruCols);
}

cudaError_t lru_forward(const LruArgs& args, const LruTensors& t, void* y, float* h_final, float* kept, void* workspace,
                        cudaStream_t s) {
    Lru p = lru_of(args, t);
    p.vec = lru_pairs(y, args.D, args.io == GDR_F32 ? 4 : 2);
    LruChain chain;
    if (cudaError_t e = lru_chain(args, workspace, &chain, s)) return e;
    return lru_types(args.io, t.lam, t.i.p, [&](auto io, auto rate, auto gate) {
        using IO = decltype(io);
        constexpr bool R = decltype(rate)::value, G = decltype(gate)::value;
        constexpr int bytes = lru_forward_smem<IO, G>();
        const auto kernel = lru_forward_kernel<IO, R, G>;
        if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) return e;
        kernel<<<std::min(p.tiles * p.cols, (unsigned)(kBlocks * kSms)), kLruThreads, bytes, s>>>(p, chain, (IO*)y, kept, h_final);
        return cudaGetLastError();
    });
}

cudaError_t lru_step(const LruArgs& args, const LruTensors& t, int64_t pool, const int* slots, float* h, void* y,
                     cudaStream_t s) {
    Lru p = lru_of(args, t);
    p.vec = lru_pairs(y, args.D, args.io == GDR_F32 ? 4 : 2);
    const dim3 grid((unsigned)((args.D + 255) / 256), (unsigned)std::min<int64_t>(args.n, 65535));
    return lru_types(args.io, t.lam, t.i.p, [&](auto io, auto rate, auto gate) {
        using IO = decltype(io);
        lru_step_kernel<IO, decltype(rate)::value, decltype(gate)::value>
            <<<grid, 128, 0, s>>>(p, args.n, pool, slots, h, (IO*)y);
        return cudaGetLastError();
    });
}

}  // namespace layer
}  // namespace gdr
