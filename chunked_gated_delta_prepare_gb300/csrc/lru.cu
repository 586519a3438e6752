// The gated linear recurrence over prompts and batches, and its single-token step (formulas in lru.cuh).
//
// Bound: memory.  One pass: a tile's rows arrive in shared memory while the block works on the tile before, a thread forms
// the decays a and terms u of its run of 8 tokens in registers, the runs' maps h -> h * decay + own are joined through
// shared memory, the tile's state comes from the tiles before it (look_back), and the run is gone over again from its state.
//
// Measured (bf16, both gates): 32768 x 4096 in 205 us, 5.2 TB/s, 0.77 of a copy's rate; with rates above 1/4 236, without
// rates 195.  What is left is the wait for a tile's state: 3.9 of 10 warps an issue stand at the group's barrier, and the issue
// slots are 0.56 full.  Blocks of one group that all look back through the L2 took 239, tiles fetched by the workers' own loads
// 286, gates by a reciprocal and a root each (see lru.cuh) 254.  Rows that TMA cannot take: 8192 x 4094 94 us, 4095 (by
// elements) 132, 4096 62.
// A step of 256 x 8192 fp16: 6.2 us, 4.8 TB/s; of 16 rows, the host's call.
#include "lru.cuh"

namespace gdr {
namespace layer {
namespace {

struct alignas(16) Map {     // what a run of tokens makes of state h: h * decay + own
    F2 decay, own;
};

// The decays and terms of the thread's run, from shared memory; a = 1, u = 0 past the tile's end.
template <typename IO, bool RATE, bool GATE>
__device__ __forceinline__ void read_run(const IO* from, int row, int pair, F2 k, F2 root, bool far, int len, int left,
                                         F2 (&a)[kLruRun], F2 (&u)[kLruRun]) {
    constexpr int N = kLruTile * kLruCols;
    RawN<IO, 2> r[kLruRun], i[kLruRun];
#pragma unroll
    for (int j = 0; j < kLruRun; ++j) {
        r[j] = lru_raw(from, row + j, pair);
        if (GATE) i[j] = lru_raw(from + 2 * N, row + j, pair);
    }
    const F2 k2 = add2(k, k);
    const auto run = [&](auto more, auto wild) {
        constexpr bool MORE = decltype(more)::value, WILD = decltype(wild)::value;
#pragma unroll
        for (int j = 0; j < kLruRun; ++j) {
            const F2 x = lru_read(from + N, row + j, pair), rv = wide2(r[j]), t2 = GATE ? one_and_exp(wide2(i[j])) : 0;
            if (RATE) {
                F2 w, z;
                lru_roots<GATE, WILD>(one_and_exp(rv), t2, w, z);
                const F2 v = mul2(k2, mul2(w, w));
                a[j] = ex2_2(fma2(v, both(-0.5f * kLog2e), both(kLruLean)));
                u[j] = mul2(mul2(z, lru_p(v)), mul2(root, x));
                if (MORE) {
                    const F2 s = sqrt2(fma2(mul2(a[j], both(-1.f)), a[j], both(1.f)));
                    u[j] = below(v, kLruNear, u[j], mul2(s, GATE ? mul2(rcp_2(t2), x) : x));
                }
            } else {
                F2 s, sg;
                lru_parts<GATE, MORE>(rv, t2, a[j], s, sg);
                u[j] = mul2(sg, x);
            }
        }
    };
    const bool tame = lru_tame<RATE, RATE && GATE>(r, i, len - row, left);
    if (tame && !(RATE && far)) run(std::false_type(), std::false_type());
    else if (RATE && tame) run(std::true_type(), std::false_type());
    else run(std::true_type(), std::bool_constant<RATE>());
    if (len < kLruTile)
#pragma unroll
        for (int j = 0; j < kLruRun; ++j)
            if (row + j >= len) a[j] = both(1.f), u[j] = both(0.f);
}

constexpr int kGroups = 3;   // 72 registers a thread
template <typename IO> constexpr int kBuffers = sizeof(IO) == 2 ? 2 : 1;      // of tiles

template <typename IO, bool GATE> constexpr int lru_forward_smem() {      // of a group
    return kBuffers<IO> * (GATE ? 3 : 2) * kLruTile * kLruCols * (int)sizeof(IO);
}

// y, kept and h_final may each be nullptr.
template <typename IO, bool RATE, bool GATE, bool TMA>
__global__ void __launch_bounds__(kGroups * kLruThreads, 1)
lru_forward_kernel(Lru p, LruChain chain, const __grid_constant__ LruMaps in_maps, IO* __restrict__ y,
                   float* __restrict__ kept, float* __restrict__ h_final) {
    constexpr int B = kBuffers<IO>, N = kLruTile * kLruCols, IN = GATE ? 3 : 2;
    struct Group {
        Map maps[kLruWarps][kLruPairs], fronts[kLruWarps][kLruPairs];      // of a warp's tokens, of those in front of them
        F2 carry[kLruPairs];
        LruPlan plans[kLruPlans];
        LruHand hand;                                       // to the next group
        uint64_t ready, full[B];                            // the tile's maps are there; its inputs are
    };
    extern __shared__ __align__(128) uint4 smem[];
    __shared__ Group all_groups[kGroups];
    const int group = threadIdx.x / kLruThreads, thread = threadIdx.x - group * kLruThreads;
    Group& me = all_groups[group];
    LruPlan* plans = me.plans;
    IO* in = reinterpret_cast<IO*>(smem) + group * (B * IN * N);           // [B][IN][N]: r, x, i

    const auto issue = [&](unsigned turn) {                 // one lane asks for a tile
        if (TMA && plans[turn % kLruPlans].live) {
            const LruTile& t = plans[turn % kLruPlans].t;
            uint64_t* bar = me.full + turn % B;
            IO* to = in + (turn % B) * IN * N;
            if (t.len == 0) return bw::mbar_arrive(bar);
            bw::mbar_arrive_expect_tx(bar, (unsigned)(IN * N * sizeof(IO)));
            lru_tma(to, &in_maps.r, bar, t);
            lru_tma(to + N, &in_maps.x, bar, t);
            if (GATE) lru_tma(to + 2 * N, &in_maps.i, bar, t);
        }
    };
    if (thread >= kLruWorkers) {                            // the guide
        const int lane = thread - kLruWorkers, pair = lane % kLruPairs;
        const bool first = lane < kLruPairs;                // the warp's other half only looks on
        if (lane == 0) {
            bw::mbar_init(&me.ready, kLruWarps);
            bw::mbar_init(&me.hand.given, 1);
            bw::mbar_init(&me.hand.taken, 1);
            for (int i = 0; i < B; ++i) bw::mbar_init(me.full + i, 1);
            bw::fence_mbar_init();
        }
        LruPlanner<false, RATE, kGroups> planner;
        planner.read(p, chain, 0);
        for (unsigned turn = 0; turn < 3; ++turn) planner.plan(p, chain, turn, group, plans + turn);
        for (unsigned turn = 0; turn < B; ++turn)
            if (lane == 0) issue(turn);
        __syncthreads();
        for (unsigned turn = 0; plans[turn % kLruPlans].live; ++turn) {
            const LruTile t = plans[turn % kLruPlans].t;
            const int ch = t.col * kLruCols + pair * 2, left = p.D - ch;
            const int64_t at = ((int64_t)t.number * p.cols + t.col) * kLruPairs + pair;
            F2 state = 0;
            bool found = t.to_head == 0, there = false;
            if (found && t.seq >= 0) state = state2(p.h0, (int64_t)t.seq * p.D + ch, left);
            if (group == 0)                                 // another block's state may be there before the tile's maps are
                while (!found && !there) {
                    found = look_back<false>(chain, t, p.cols, pair, t.to_head, state);
                    there = __all_sync(0xffffffffu, bw::mbar_test_wait(&me.ready, turn & 1));
                }
            if (!there) bw::mbar_wait(&me.ready, turn & 1, chain.err, kDeviceErrTimeout);
            Map m[kLruWarps], all{both(1.f), both(0.f)};
#pragma unroll
            for (int w = 0; w < kLruWarps; ++w) m[w] = me.maps[w][pair];
#pragma unroll
            for (int w = 0; w < kLruWarps; ++w) {
                if (first) me.fronts[w][pair] = all;
                all.own = fma2(m[w].decay, all.own, m[w].own);
                all.decay = mul2(m[w].decay, all.decay);
            }
            if (first && t.to_tail && t.to_head) publish_map(chain.maps + at, all.decay, all.own);
            if (group == 0) {
                if (!found) state = wait_back<false>(chain, t, p.cols, pair, t.to_head);
            } else if (chain.maps) {
                const F2 given = lru_take(all_groups[group - 1].hand, turn, chain.err);
                if (!found) state = given;
            }
            const F2 end = fma2(all.decay, state, all.own);
            if (first) me.carry[pair] = state;
            lru_arrive<2, kLruThreads>(group);
            if (group + 1 < kGroups && chain.maps) lru_give(me.hand, end, turn, chain.err);
            if (first && t.to_tail) publish_state(chain.states + at + (int64_t)p.cols * kLruPairs, end);
            if (first && t.seq >= 0) {
                if (kept) put_state2(kept, (int64_t)t.number * p.D + ch, state, left);
                if (h_final && !t.to_tail) put_state2(h_final, (int64_t)t.seq * p.D + ch, end, left);
            }
            planner.plan(p, chain, turn + 3, group, plans + (turn + 3) % kLruPlans);
        }
        return;
    }

    const int warp = thread / 32, pair = thread % kLruPairs, row = thread / kLruPairs * kLruRun;
    const bool second = thread & 16;                        // run of the warp
    const auto fetch = [&](unsigned turn) {
        if (plans[turn % kLruPlans].live) {
            const LruTile t = plans[turn % kLruPlans].t;
            IO* to = in + (turn % B) * IN * N;
            lru_fetch(p.r, t, p.D, thread, to);
            lru_fetch(p.x, t, p.D, thread, to + N);
            if (GATE) lru_fetch(p.i, t, p.D, thread, to + 2 * N);
        }
        copy_group();
    };
    __syncthreads();
    if (!TMA)
        for (unsigned turn = 0; turn < B; ++turn) fetch(turn);
    for (unsigned turn = 0; plans[turn % kLruPlans].live; ++turn) {
        if (TMA) {
            bw::mbar_wait(me.full + turn % B, turn / B & 1, chain.err, kDeviceErrTimeout);
        } else {
            copy_wait<B - 1>();
            lru_sync<1, kLruWorkers>(group);
        }
        const LruPlan& plan = plans[turn % kLruPlans];
        const int len = plan.t.len, ch = plan.t.col * kLruCols + pair * 2, left = p.D - ch;
        const bool some = warp * 2 * kLruRun < len;         // short sequences leave warps without a token: 2000 of 16 x 4096
                                                            // take half the time of going through them all
        F2 a[kLruRun], u[kLruRun];
        Map m{both(1.f), both(0.f)};
        if (some) {
            F2 k = 0, root = 0;
            if (RATE) {
                k = *reinterpret_cast<const F2*>(plan.rates + pair * 2);
                root = *reinterpret_cast<const F2*>(plan.roots + pair * 2);
            }
            read_run<IO, RATE, GATE>(in + (turn % B) * IN * N, row, pair, k, root, plan.far, len, left, a, u);
            m = Map{a[0], u[0]};
#pragma unroll
            for (int j = 1; j < kLruRun; ++j) {
                m.own = fma2(a[j], m.own, u[j]);
                m.decay = mul2(a[j], m.decay);
            }
        }
        Map o{swap_halves(m.decay), swap_halves(m.own)};    // of the warp's other run
        if (!second) me.maps[warp][pair] = Map{mul2(o.decay, m.decay), fma2(o.decay, m.own, o.own)};
        __syncwarp();
        if ((thread & 31) == 0) bw::mbar_arrive(&me.ready);
        lru_sync<2, kLruThreads>(group);
        if (!TMA) fetch(turn + B);
        else if (thread == kLruWorkers - 32) issue(turn + B);
        if (y && some) {
            F2 h = fma2(me.fronts[warp][pair].decay, me.carry[pair], me.fronts[warp][pair].own);
            if (second) h = fma2(o.decay, h, o.own);
            IO* yp = y + (plan.t.first + row) * p.D + ch;
            if (p.vec && len == kLruTile && left > 0) {
#pragma unroll
                for (int j = 0; j < kLruRun; ++j) {
                    h = fma2(a[j], h, u[j]);
                    store2(yp, h, 2, true);
                    yp += p.D;
                }
            } else {
#pragma unroll
                for (int j = 0; j < kLruRun; ++j) {
                    h = fma2(a[j], h, u[j]);
                    if (row + j < len) store2(yp, h, left, false);
                    yp += p.D;
                }
            }
        }
    }
}

__global__ void __launch_bounds__(256)
lru_chain_kernel(uint4* __restrict__ words, int64_t n, const float* __restrict__ lam, float c, int D,
                 float4* __restrict__ rates, int channels) {
    const int64_t step = (int64_t)gridDim.x * 256, at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    for (int64_t i = at; i < n; i += step) words[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
    if (lam)
        for (int64_t ch = at; ch < channels; ch += step) rates[ch] = ch < D ? rates_of(lam[ch], c) : float4{};
}

// A thread takes four neighbouring channels of a row; quads: whole vectors of them are aligned in every tensor.
template <typename IO, bool RATE, bool GATE>
__global__ void __launch_bounds__(128)
lru_step_kernel(Lru p, int64_t rows, int64_t pool, const int* __restrict__ slots, float* __restrict__ h, IO* __restrict__ y,
                bool quads) {
    const int ch = (blockIdx.x * 128 + threadIdx.x) * 4, left = p.D - ch;
    if (left <= 0) return;
    F2 k[2] = {0, 0};
    if (RATE) {
        const auto rate = [&](int c) { return c < left ? rate_of(p.lam[ch + c], p.c) : 0.f; };
        k[0] = pack2(rate(0), rate(1)), k[1] = pack2(rate(2), rate(3));
    }
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        const int64_t slot = slots ? slots[row] : row;
        const bool some = slot >= 0 && slot < pool;
        float* hp = h + slot * p.D + ch;
        float out[4] = {0.f, 0.f, 0.f, 0.f};
        if (some) {
            const auto in = [&](const LruRows& v) { return load_n<4>((const IO*)v.p + row * v.ld + ch, left, quads); };
            const RawN<IO, 4> r = in(p.r), x = in(p.x), i = GATE ? in(p.i) : r;
            const RawN<float, 4> old = load_own<4>(hp, left, quads);
            F2 rv[2], xv[2], iv[2];
            pairs<IO, 4>(r, rv), pairs<IO, 4>(x, xv), pairs<IO, 4>(i, iv);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                F2 a, s, q;
                decay_and_part<RATE>(rv[c], k[c], a, s, q);
                F2 u = mul2(s, xv[c]);
                if (GATE) u = mul2(u, sigmoid2(iv[c]));
                const float2 n = unpack2(fma2(a, pack2(old.e[2 * c], old.e[2 * c + 1]), u));
                out[2 * c] = n.x, out[2 * c + 1] = n.y;
            }
            store_n(hp, out, left, quads);
        }
        store_n(y + row * p.D + ch, out, left, quads);
    }
}

}  // namespace

int64_t lru_tiles(const LruArgs& a) { return tile_count(Seqs{a.cu, a.total, a.T, (int)a.n}, kLruTile); }

size_t lru_forward_workspace(const LruArgs& a) {
    return lru_one_tile_each(a) ? 0 : lru_chain_bytes(lru_tiles(a), (a.D + kLruCols - 1) / kLruCols);
}

cudaError_t lru_chain(const LruArgs& a, const float* lam, void* workspace, LruChain* c, cudaStream_t s) {
    *c = LruChain{};
    if (cudaError_t e = device_error_ptr(&c->err)) return e;
    if (lru_one_tile_each(a)) return cudaSuccess;
    const int64_t cols = (a.D + kLruCols - 1) / kLruCols, cells = lru_tiles(a) * cols * kLruPairs;
    c->maps = (ulonglong2*)workspace;
    c->states = (F2*)(c->maps + cells);
    float4* rates = (float4*)(c->states + cells);
    c->rates = lam ? rates : nullptr;
    const int64_t n = cells * 24 / 16;                     // 16 bytes each
    lru_chain_kernel<<<(unsigned)std::min<int64_t>((n + 1023) / 1024, 8 * kSms), 256, 0, s>>>(
        (uint4*)workspace, n, lam, a.c, a.D, rates, (int)(cols * kLruCols));
    return cudaGetLastError();
}

cudaError_t lru_forward(const LruArgs& args, const LruTensors& t, void* y, float* h_final, float* kept, void* workspace,
                        cudaStream_t s) {
    Lru p = lru_of(args, t, kGroups);
    p.vec = lru_pairs(y, args.D, args.io == GDR_F32 ? 4 : 2);
    LruChain chain;
    if (cudaError_t e = lru_chain(args, t.lam, workspace, &chain, s)) return e;
    LruMaps m;
    const bool tma = args.total > 0 && p.x.unit == 16 && p.r.unit == 16 && (!p.i.p || p.i.unit == 16);
    if (tma && !(lru_map(&m.x, p.x, args) && lru_map(&m.r, p.r, args) && (!p.i.p || lru_map(&m.i, p.i, args))))
        return cudaErrorInvalidValue;
    return lru_types(args.io, t.lam, t.i.p, [&](auto io, auto rate, auto gate) {
        using IO = decltype(io);
        constexpr bool R = decltype(rate)::value, G = decltype(gate)::value;
        const auto go = [&](auto kernel) {
            return lru_launch(kernel, p, chain, kGroups * kLruThreads, kGroups * lru_forward_smem<IO, G>(), s, m, (IO*)y, kept,
                              h_final);
        };
        return tma ? go(lru_forward_kernel<IO, R, G, true>) : go(lru_forward_kernel<IO, R, G, false>);
    });
}

cudaError_t lru_step(const LruArgs& args, const LruTensors& t, int64_t pool, const int* slots, float* h, void* y,
                     cudaStream_t s) {
    const Lru p = lru_of(args, t, kGroups);
    const int64_t e = args.io == GDR_F32 ? 4 : 2;
    bool quads = args.D % 4 == 0 && reinterpret_cast<uintptr_t>(h) % 16 == 0 && reinterpret_cast<uintptr_t>(y) % (4 * e) == 0;
    for (const LruRows* v : {&p.x, &p.r, &p.i})
        quads = quads && reinterpret_cast<uintptr_t>(v->p) % (4 * e) == 0 && (!v->p || v->ld % 4 == 0);
    const dim3 grid((unsigned)((args.D + 511) / 512), (unsigned)std::min<int64_t>(args.n, 65535));
    return lru_types(args.io, t.lam, t.i.p, [&](auto io, auto rate, auto gate) {
        using IO = decltype(io);
        lru_step_kernel<IO, decltype(rate)::value, decltype(gate)::value>
            <<<grid, 128, 0, s>>>(p, args.n, pool, slots, h, (IO*)y, quads);
        return cudaGetLastError();
    });
}

}  // namespace layer
}  // namespace gdr
