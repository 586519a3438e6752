// The gated linear recurrence over prompts and batches, and its single-token step (formulas in lru.cuh).
//
// Bound: memory.  A tile of 128 tokens by 64 channels is a block's: warp w takes the tokens 8 w .. 8 w + 7, forms their
// decays a and terms u in registers, and from a zero state the run's last state and product of decays; a thread then
// folds the runs in front of its own, from the tile's first state, through shared memory and goes over its run again.
// The states in front of the tiles come from two kernels before: the tiles' own ends, and a serial pass over them.
#include "lru.cuh"

namespace gdr {
namespace layer {
namespace {

struct alignas(16) End {     // of a run of tokens: what it makes of state h is h * decay + own
    F2 decay, own;
};

// The decays and terms of the thread's tokens; a = 1, u = 0 past the tile's end.
template <typename IO, bool RATE, bool GATE>
__device__ __forceinline__ void load_run(const Lru& p, const LruTile& t, int t0, const Rate& k, F2 (&a)[kLruTokens],
                                         F2 (&u)[kLruTokens]) {
    RawN<IO, 2> x[kLruTokens], r[kLruTokens], i[kLruTokens];
    const int64_t row = t.first + t0;
    const IO* xp = (const IO*)p.x.p + row * p.x.ld + t.ch;
    const IO* rp = (const IO*)p.r.p + row * p.r.ld + t.ch;
    const IO* ip = (const IO*)p.i.p + row * p.i.ld + t.ch;
#pragma unroll
    for (int j = 0; j < kLruTokens; ++j) {
        if (t0 + j >= t.len) continue;
        r[j] = load2(rp + j * p.r.ld, t.left, p.r.vec);
        x[j] = load2(xp + j * p.x.ld, t.left, p.x.vec);
        if (GATE) i[j] = load2(ip + j * p.i.ld, t.left, p.i.vec);
    }
#pragma unroll
    for (int j = 0; j < kLruTokens; ++j) {
        if (t0 + j >= t.len) {
            a[j] = both(1.f), u[j] = both(0.f);
            continue;
        }
        F2 s;
        decay_and_part<RATE>(wide2(r[j]), k, a[j], s);
        u[j] = mul2(s, wide2(x[j]));
        if (GATE) u[j] = mul2(u[j], sigmoid2(wide2(i[j])));
    }
}

__device__ __forceinline__ End end_of(const F2 (&a)[kLruTokens], const F2 (&u)[kLruTokens]) {
    End e{a[0], u[0]};
#pragma unroll
    for (int j = 1; j < kLruTokens; ++j) {
        e.own = fma2(a[j], e.own, u[j]);
        e.decay = mul2(a[j], e.decay);
    }
    return e;
}

// The tiles' ends [tiles][D]: decay, own.
template <typename IO, bool RATE, bool GATE>
__global__ void __launch_bounds__(kLruWarps * 32) lru_ends_kernel(Lru p, float2* __restrict__ ends) {
    __shared__ End run[kLruWarps][32];
    const LruTile t = lru_tile(p, blockIdx.x);
    if (t.seq < 0 || t.tail) return;                   // nobody goes on from a sequence's last tile
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Rate k{0, 0};
    if (RATE) k = load_rate(p, t.ch, false);
    F2 a[kLruTokens], u[kLruTokens];
    load_run<IO, RATE, GATE>(p, t, warp * kLruTokens, k, a, u);
    run[warp][lane] = end_of(a, u);
    __syncthreads();
    if (warp) return;
    End e = run[0][lane];
#pragma unroll
    for (int w = 1; w < kLruWarps; ++w) {
        const End n = run[w][lane];
        e.own = fma2(n.decay, e.own, n.own);
        e.decay = mul2(n.decay, e.decay);
    }
    const float2 d = unpack2(e.decay), o = unpack2(e.own);
    float2* out = ends + t.number * p.D + t.ch;
    if (t.left > 0) out[0] = make_float2(d.x, o.x);
    if (t.left > 1) out[1] = make_float2(d.y, o.y);
}

// The state in front of every tile, a thread a channel of a sequence.
__global__ void __launch_bounds__(64) lru_join_kernel(Lru p, const float2* __restrict__ ends, float* __restrict__ kept) {
    const int ch = blockIdx.x * 64 + threadIdx.x;
    if (ch >= p.D) return;
    for (int s = blockIdx.y; s < p.q.n; s += gridDim.y) {
        int64_t start, len;
        seq_range(p.q, s, &start, &len);
        const int64_t first = first_tile(p.q, s, kLruTile), tiles = (len + kLruTile - 1) / kLruTile;
        float h = p.h0 ? p.h0[(int64_t)s * p.D + ch] : 0.f;
        kept[first * p.D + ch] = h;
#pragma unroll 8
        for (int64_t i = 0; i + 1 < tiles; ++i) {
            const float2 e = ends[(first + i) * p.D + ch];
            h = fmaf(e.x, h, e.y);
            kept[(first + i + 1) * p.D + ch] = h;
        }
    }
}

// kept: the states in front of the tiles (nullptr: every sequence is one tile, and starts from h0).
template <typename IO, bool RATE, bool GATE>
__global__ void __launch_bounds__(kLruWarps * 32)
lru_forward_kernel(Lru p, const float* __restrict__ kept, IO* __restrict__ y, float* __restrict__ h_final) {
    __shared__ End run[kLruWarps][32];
    const LruTile t = lru_tile(p, blockIdx.x);
    if (t.seq < 0) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t0 = warp * kLruTokens;
    F2 h = kept ? state2(kept, t.number * p.D + t.ch, t.left) : state2(p.h0, (int64_t)t.seq * p.D + t.ch, t.left);
    Rate k{0, 0};
    if (RATE) k = load_rate(p, t.ch, false);
    F2 a[kLruTokens], u[kLruTokens];
    load_run<IO, RATE, GATE>(p, t, t0, k, a, u);
    run[warp][lane] = end_of(a, u);
    __syncthreads();
    for (int w = 0; w < warp; ++w) h = fma2(run[w][lane].decay, h, run[w][lane].own);
    IO* yp = y + (t.first + t0) * p.D + t.ch;
#pragma unroll
    for (int j = 0; j < kLruTokens; ++j) {
        h = fma2(a[j], h, u[j]);
        if (t0 + j < t.len) store2(yp + (int64_t)j * p.D, h, t.left, p.vec);
    }
    if (h_final && t.tail && warp == kLruWarps - 1)      // past the end the state stays what it is
        put_state2(h_final, (int64_t)t.seq * p.D + t.ch, h, t.left);
}

template <typename IO, bool RATE, bool GATE>
__global__ void __launch_bounds__(128)
lru_step_kernel(Lru p, int64_t rows, int64_t pool, const int* __restrict__ slots, float* __restrict__ h, IO* __restrict__ y) {
    const int ch = (blockIdx.x * 128 + threadIdx.x) * 2, left = p.D - ch;
    if (left <= 0) return;
    Rate k{0, 0};
    if (RATE) k = load_rate(p, ch, false);
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        const int64_t slot = slots ? slots[row] : row;
        IO* yp = y + row * p.D + ch;
        if (slot < 0 || slot >= pool) {
            store2(yp, both(0.f), left, p.vec);
            continue;
        }
        F2 a, s;
        decay_and_part<RATE>(wide2(load2((const IO*)p.r.p + row * p.r.ld + ch, left, p.r.vec)), k, a, s);
        F2 u = mul2(s, wide2(load2((const IO*)p.x.p + row * p.x.ld + ch, left, p.x.vec)));
        if (GATE) u = mul2(u, sigmoid2(wide2(load2((const IO*)p.i.p + row * p.i.ld + ch, left, p.i.vec))));
        const F2 n = fma2(a, state2(h, slot * p.D + ch, left), u);
        put_state2(h, slot * p.D + ch, n, left);
        store2(yp, n, left, p.vec);
    }
}

bool one_tile_each(const LruArgs& a) { return (a.cu ? a.total : a.T) <= kLruTile; }

}  // namespace

int64_t lru_tiles(const LruArgs& a) { return tile_count(Seqs{a.cu, a.total, a.T, (int)a.n}, kLruTile); }

size_t lru_forward_workspace(const LruArgs& a, bool kept) {
    if (one_tile_each(a)) return 0;
    return (size_t)lru_tiles(a) * a.D * (kept ? 8 : 12);
}

// The states in front of all tiles.
cudaError_t lru_states(const LruArgs& args, const LruTensors& t, float2* ends, float* kept, cudaStream_t s) {
    const Lru p = lru_of(args, t);
    if (!one_tile_each(args)) {
        const cudaError_t e = lru_types(args.io, t.lam, t.i.p, [&](auto io, auto rate, auto gate) {
            lru_ends_kernel<decltype(io), decltype(rate)::value, decltype(gate)::value>
                <<<(unsigned)(lru_tiles(args) * p.cols), kLruWarps * 32, 0, s>>>(p, ends);
            return cudaGetLastError();
        });
        if (e != cudaSuccess) return e;
    }
    const dim3 grid((unsigned)((args.D + 63) / 64), (unsigned)std::min<int64_t>(args.n, 65535));
    lru_join_kernel<<<grid, 64, 0, s>>>(p, ends, kept);
    return cudaGetLastError();
}

cudaError_t lru_forward(const LruArgs& args, const LruTensors& t, void* y, float* h_final, float* kept, float* workspace,
                        cudaStream_t s) {
    Lru p = lru_of(args, t);
    p.vec = lru_pairs(y, args.D, args.io == GDR_F32 ? 4 : 2);
    float2* ends = (float2*)workspace;
    if (!kept && !one_tile_each(args)) kept = workspace + lru_tiles(args) * args.D * 2;
    if (kept)
        if (cudaError_t e = lru_states(args, t, ends, kept, s)) return e;
    return lru_types(args.io, t.lam, t.i.p, [&](auto io, auto rate, auto gate) {
        using IO = decltype(io);
        lru_forward_kernel<IO, decltype(rate)::value, decltype(gate)::value>
            <<<(unsigned)(lru_tiles(args) * p.cols), kLruWarps * 32, 0, s>>>(p, kept, (IO*)y, h_final);
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
