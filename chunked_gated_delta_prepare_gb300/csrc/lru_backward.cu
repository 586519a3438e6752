// The gradient of the gated linear recurrence (formulas in lru.cuh).  With e_t the gradient of h_t:
//
//   e_t = dy_t + a_{t+1} e_{t+1}   (the last: + dh_final),   dh0 = a_1 e_1
//   dx = e s g,  di = e s x g (1 - g)
//   RATE:  dlog a = e a (h_{t-1} - g x a / s),  dr = -dlog a k q (1 - q),  dlam = -sum dlog a q c sigmoid(lam)
//   else:  dr = e a s (h_{t-1} - g x)
//
// Bound: memory, and (at 18 warps an SM) the latency of what a tile waits for in turn: its inputs, the gradient from behind,
// its outputs.  One pass over the tiles from behind: as in the forward, with the gradient that reaches a tile from behind in
// the place of its state, which is the forward's kept one.  Two groups a block: of three neither the registers (72 a thread, of
// which a run's a, h and s take 48) nor, with gates, the shared memory would hold the work.
//
// Measured (bf16, both gates, kept states): 4 x 2048 x 4096 in 110 us, 4.3 TB/s, 0.63 of a copy's rate; issue slots 0.52 full
// with 4.5 warps in each to choose from.  With the gates' products formed token by token, with 64-bit offsets and reciprocals
// of their own it took 130.  With rates above 1/4, 8192 x 4096: 156 us (120 below); without rates 98.
#include "lru.cuh"

namespace gdr {
namespace layer {
namespace {

constexpr int kGroups = 2;   // 96 registers a thread
template <typename IO> constexpr int kBuffers = sizeof(IO) == 2 ? 2 : 1;      // of tiles

// A token's e^-i, and (RATE) (1 - q) / 2, wait in shared memory while the tile's maps are joined: in registers, beside the run's
// a, h and s, they spill (4 x 2048 x 4096 bf16 133 us, so 120).  They lie in room of their own behind the tiles, a number of a
// thread's token j at [j][thread]; but without TMA, where rows come through the L1 that this room is taken from, the second
// lies in the place of its r (16-bit types: of its r and its i), which no other thread reads (8192 x 4094 226 us otherwise, so
// 191).
template <bool RATE, bool GATE, bool TMA> constexpr bool kHalfBehind = RATE && (TMA || !GATE);
constexpr int kAside = kLruRun * kLruWorkers;
template <typename IO, bool RATE, bool GATE, bool TMA> struct Aside {
    static constexpr int numbers = kHalfBehind<RATE, GATE, TMA> + GATE;
    F2* room;                // the thread's
    IO* place;               // the tile

    __device__ __forceinline__ F2& shut(int j) const { return room[kHalfBehind<RATE, GATE, TMA> * kAside + j * kLruWorkers]; }
    __device__ __forceinline__ void put_half(int j, int row, int pair, F2 v) const {
        IO* const at = place + (row + j) * kLruCols + pair * 2;
        if constexpr (kHalfBehind<RATE, GATE, TMA>) {
            room[j * kLruWorkers] = v;
        } else if constexpr (sizeof(IO) == 4) {
            *reinterpret_cast<F2*>(at) = v;
        } else {
            const float2 f = unpack2(v);
            *reinterpret_cast<float*>(at) = f.x;
            *reinterpret_cast<float*>(at + 3 * kLruTile * kLruCols) = f.y;
        }
    }
    __device__ __forceinline__ F2 half(int j, int row, int pair) const {
        const IO* const at = place + (row + j) * kLruCols + pair * 2;
        if constexpr (kHalfBehind<RATE, GATE, TMA>) return room[j * kLruWorkers];
        else if constexpr (sizeof(IO) == 4) return *reinterpret_cast<const F2*>(at);
        else return pack2(*reinterpret_cast<const float*>(at), *reinterpret_cast<const float*>(at + 3 * kLruTile * kLruCols));
    }
};
template <typename IO, bool RATE, bool GATE, bool TMA> constexpr int lru_backward_smem() {     // of a group
    return kBuffers<IO> * (GATE ? 4 : 3) * kLruTile * kLruCols * (int)sizeof(IO) +
           Aside<IO, RATE, GATE, TMA>::numbers * kAside * (int)sizeof(F2);
}

struct alignas(8) Run {      // of a run of tokens: its product of decays, its end from a zero state, and what it sends to the
    F2 decay, own, back;     // state before it with nothing behind it
};
struct alignas(16) Map {     // what tokens make of the gradient e from behind them: e * decay + back
    F2 decay, back;
};

__device__ __forceinline__ F2 at_most(F2 v, float bound) {
    const float2 f = unpack2(v);
    return pack2(min_nan(f.x, bound), min_nan(f.y, bound));
}

// The decays and terms of the thread's run, from shared memory, and what the gradients need beside them: the input's part s
// (RATE: sqrt(v), v = 2 k q), and what is set aside.  1 - q and 1 - g = e^-i g come from the exponentials: from q and g, which
// are rounded, an open gate's would be noise.  RATE: the terms, and so all states here, have the other sign, which saves the
// gradients a negation.  A token past the tile's end has a = 1, u = 0.
template <typename IO, bool RATE, bool GATE, bool TMA>
__device__ __forceinline__ void read_run(const Aside<IO, RATE, GATE, TMA>& aside, int row, int pair, F2 root, bool far, int len,
                                         int left, F2 (&a)[kLruRun], F2 (&u)[kLruRun], F2 (&part)[kLruRun]) {
    const IO* const from = aside.place;
    constexpr int N = kLruTile * kLruCols;
    RawN<IO, 2> r[kLruRun], i[kLruRun];
#pragma unroll
    for (int j = 0; j < kLruRun; ++j) {
        r[j] = lru_raw(from, row + j, pair);
        if (GATE) i[j] = lru_raw(from + 3 * N, row + j, pair);
    }
    const F2 minus = neg2(root);
    const auto run = [&](auto more, auto wild) {
        constexpr bool MORE = decltype(more)::value, WILD = decltype(wild)::value;
#pragma unroll
        for (int j = 0; j < kLruRun; ++j) {
            const F2 x = lru_read(from + N, row + j, pair), rv = wide2(r[j]);
            const F2 e = GATE ? ex2_2(mul2(wide2(i[j]), both(-kLog2e))) : 0;
            if (RATE) {
                F2 w, z;
                const F2 half = ex2_2(fma2(rv, both(-kLog2e), both(-1.f)));         // e^-r / 2
                lru_roots<GATE, WILD>(fma2(half, both(2.f), both(1.f)), add2(e, both(1.f)), w, z);
                part[j] = mul2(root, w);
                const F2 v = mul2(part[j], part[j]);
                a[j] = ex2_2(fma2(v, both(-0.5f * kLog2e), both(kLruLean)));
                u[j] = mul2(mul2(z, lru_p(v)), mul2(minus, x));
                if (MORE) {
                    const F2 s = sqrt2(fma2(mul2(a[j], both(-1.f)), a[j], both(1.f)));
                    u[j] = below(v, kLruNear, u[j], mul2(neg2(s), GATE ? mul2(rcp_2(add2(e, both(1.f))), x) : x));
                }
                aside.put_half(j, row, pair, mul2(at_most(half, kLruHuge), mul2(w, w)));
            } else {
                F2 sg;
                lru_parts<GATE, MORE>(rv, add2(e, both(1.f)), a[j], part[j], sg);
                u[j] = mul2(sg, x);
            }
            if (GATE) aside.shut(j) = WILD || (MORE && !RATE) ? at_most(e, kLruHuge) : e;
        }
    };
    const bool tame = lru_tame<RATE, GATE>(r, i, len - row, left);
    if (tame && !(RATE && far)) run(std::false_type(), std::false_type());
    else if (RATE && tame) run(std::true_type(), std::false_type());
    else run(std::true_type(), std::bool_constant<RATE>());
    if (len < kLruTile)
#pragma unroll
        for (int j = 0; j < kLruRun; ++j)
            if (row + j >= len) a[j] = both(1.f), u[j] = both(0.f);
}

// RATE: v = 2 k q of a token, s and v / s, the last two by P(v) where 1 - a^2 cancels: finite where s is zero.
struct Parts {
    F2 v, s, ratio;
};
__device__ __forceinline__ Parts parts_of(F2 rw, F2 a, bool far) {
    const F2 v = mul2(rw, rw);
    Parts o{v, mul2(rw, lru_p(v)), mul2(rw, lru_p_inverse(v))};
    if (far) {
        const F2 s = sqrt2(fma2(mul2(a, both(-1.f)), a, both(1.f)));
        o.s = below(v, kLruNear, o.s, s);
        o.ratio = below(v, kLruNear, o.ratio, mul2(v, rcp_2(s)));
    }
    return o;
}

// dlam: [tiles][D] partial sums, or nullptr.
template <typename IO, bool RATE, bool GATE, bool TMA>
__global__ void __launch_bounds__(kGroups * kLruThreads, 1)
lru_backward_kernel(Lru p, LruChain chain, const __grid_constant__ LruMaps in_maps, LruRows dy, const float* __restrict__ kept,
                    const float* __restrict__ dh_final, IO* __restrict__ dx, IO* __restrict__ dr, IO* __restrict__ di,
                    float* __restrict__ dlam, float* __restrict__ dh0) {
    constexpr int B = kBuffers<IO>, N = kLruTile * kLruCols, IN = GATE ? 4 : 3;
    struct Group {
        Run runs[kLruWarps][kLruPairs];                     // of a warp's tokens
        Map behind[kLruWarps][kLruPairs];                   // of the tokens behind them
        F2 fronts[kLruWarps][kLruPairs], sums[kLruWarps][kLruPairs];       // states in front of them; sums for dlam
        F2 carry[kLruPairs];
        LruPlan plans[kLruPlans];
        LruHand hand;                                       // to the next group, which has the tile before
        uint64_t ready, full[B];                            // the tile's maps are there; its inputs are
    };
    extern __shared__ __align__(128) uint4 smem[];
    __shared__ Group all_groups[kGroups];
    const int group = threadIdx.x / kLruThreads, thread = threadIdx.x - group * kLruThreads;
    Group& me = all_groups[group];
    LruPlan* plans = me.plans;
    IO* in = reinterpret_cast<IO*>(smem) + group * (B * IN * N);           // [B][IN][N]: r, x, dy, i

    const auto issue = [&](unsigned turn) {                 // one lane asks for a tile
        if (TMA && plans[turn % kLruPlans].live) {
            const LruTile& t = plans[turn % kLruPlans].t;
            uint64_t* bar = me.full + turn % B;
            IO* to = in + (turn % B) * IN * N;
            if (t.len == 0) return bw::mbar_arrive(bar);
            bw::mbar_arrive_expect_tx(bar, (unsigned)(IN * N * sizeof(IO)));
            lru_tma(to, &in_maps.r, bar, t);
            lru_tma(to + N, &in_maps.x, bar, t);
            lru_tma(to + 2 * N, &in_maps.dy, bar, t);
            if (GATE) lru_tma(to + 3 * N, &in_maps.i, bar, t);
        }
    };
    if (thread >= kLruWorkers) {                            // the guide
        const int lane = thread - kLruWorkers, pair = lane % kLruPairs;
        const bool first = lane < kLruPairs;
        if (lane == 0) {
            bw::mbar_init(&me.ready, kLruWarps);
            bw::mbar_init(&me.hand.given, 1);
            bw::mbar_init(&me.hand.taken, 1);
            for (int i = 0; i < B; ++i) bw::mbar_init(me.full + i, 1);
            bw::fence_mbar_init();
        }
        LruPlanner<true, RATE, kGroups> planner;
        planner.read(p, chain, 0);
        for (unsigned turn = 0; turn < 3; ++turn) planner.plan(p, chain, turn, group, plans + turn);
        for (unsigned turn = 0; turn < B; ++turn)
            if (lane == 0) issue(turn);
        __syncthreads();
        for (unsigned turn = 0; plans[turn % kLruPlans].live; ++turn) {
            const LruTile t = plans[turn % kLruPlans].t;
            const int ch = t.col * kLruCols + pair * 2, left = p.D - ch;
            const int64_t at = ((int64_t)t.number * p.cols + t.col) * kLruPairs + pair;
            F2 state = t.seq >= 0 ? state2(kept, (int64_t)t.number * p.D + ch, left) : 0;
            if (RATE) state = neg2(state);
            F2 e = 0;
            bool found = t.to_tail == 0, there = false;
            if (found && t.seq >= 0) e = state2(dh_final, (int64_t)t.seq * p.D + ch, left);
            if (group == 0)
                while (!found && !there) {
                    found = look_back<true>(chain, t, p.cols, pair, t.to_tail, e);
                    there = __all_sync(0xffffffffu, bw::mbar_test_wait(&me.ready, turn & 1));
                }
            if (!there) bw::mbar_wait(&me.ready, turn & 1, chain.err, kDeviceErrTimeout);
            // one half joins the gradients' maps from behind, the other the states
            F2 d = both(1.f), b = both(0.f), decay[kLruWarps], part[kLruWarps];
#pragma unroll
            for (int w = 0; w < kLruWarps; ++w) {
                decay[w] = me.runs[w][pair].decay;
                part[w] = first ? me.runs[w][pair].back : me.runs[w][pair].own;
            }
            if (first) {
#pragma unroll
                for (int w = kLruWarps - 1; w >= 0; --w) {
                    me.behind[w][pair] = Map{d, b};
                    b = fma2(decay[w], b, part[w]);
                    d = mul2(decay[w], d);
                }
            } else {
#pragma unroll
                for (int w = 0; w < kLruWarps; ++w) {
                    me.fronts[w][pair] = state;
                    state = fma2(decay[w], state, part[w]);
                }
            }
            d = __shfl_sync(0xffffffffu, d, pair);
            b = __shfl_sync(0xffffffffu, b, pair);
            if (first && t.to_head && t.to_tail) publish_map(chain.maps + at, d, b);
            if (group == 0) {
                if (!found) e = wait_back<true>(chain, t, p.cols, pair, t.to_tail);
            } else if (chain.maps) {
                const F2 given = lru_take(all_groups[group - 1].hand, turn, chain.err);
                if (!found) e = given;
            }
            const F2 end = fma2(d, e, b);
            if (first) me.carry[pair] = e;
            lru_arrive<2, kLruThreads>(group);
            if (group + 1 < kGroups && chain.maps) lru_give(me.hand, end, turn, chain.err);
            if (first && t.to_head) publish_state(chain.states + at - (int64_t)p.cols * kLruPairs, end);
            if (first && dh0 && t.seq >= 0 && !t.to_head) put_state2(dh0, (int64_t)t.seq * p.D + ch, end, left);
            planner.plan(p, chain, turn + 3, group, plans + (turn + 3) % kLruPlans);
        }
        return;
    }

    using Aside = Aside<IO, RATE, GATE, TMA>;
    F2* const room = reinterpret_cast<F2*>(reinterpret_cast<IO*>(smem) + kGroups * B * IN * N) + group * Aside::numbers * kAside +
                     thread;
    const int warp = thread / 32, pair = thread % kLruPairs, row = thread / kLruPairs * kLruRun;
    const bool second = thread & 16;                        // run of the warp
    const auto fetch = [&](unsigned turn) {
        if (plans[turn % kLruPlans].live) {
            const LruTile t = plans[turn % kLruPlans].t;
            IO* to = in + (turn % B) * IN * N;
            lru_fetch(p.r, t, p.D, thread, to);
            lru_fetch(p.x, t, p.D, thread, to + N);
            lru_fetch(dy, t, p.D, thread, to + 2 * N);
            if (GATE) lru_fetch(p.i, t, p.D, thread, to + 3 * N);
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
        const int ch = plan.t.col * kLruCols + pair * 2, left = p.D - ch, len = plan.t.len;
        const F2 root = RATE ? *reinterpret_cast<const F2*>(plan.roots + pair * 2) : 0;
        const Aside aside{room, in + (turn % B) * IN * N};
        const IO* const from = aside.place;
        F2 a[kLruRun], h[kLruRun], part[kLruRun];
        read_run(aside, row, pair, root, RATE && plan.far, len, left, a, h, part);
        Run m{both(1.f), both(0.f), both(0.f)};
#pragma unroll
        for (int j = 0; j < kLruRun; ++j) {
            m.own = fma2(a[j], m.own, h[j]);
            m.decay = mul2(m.decay, a[j]);
        }
        if (len == kLruTile) {
#pragma unroll
            for (int j = kLruRun - 1; j >= 0; --j) m.back = mul2(a[j], add2(m.back, lru_read(from + 2 * N, row + j, pair)));
        } else {
#pragma unroll
            for (int j = kLruRun - 1; j >= 0; --j)
                if (row + j < len) m.back = mul2(a[j], add2(m.back, lru_read(from + 2 * N, row + j, pair)));
        }
        // the warp's other run; the first run passes its states on, the second what it sends back
        const F2 decay = swap_halves(m.decay), other = swap_halves(second ? m.back : m.own);
        const F2 more = swap_halves(second ? m.own : m.back);
        if (!second) me.runs[warp][pair] = Run{mul2(m.decay, decay), fma2(decay, m.own, more), fma2(m.decay, other, m.back)};
        __syncwarp();
        if ((thread & 31) == 0) bw::mbar_arrive(&me.ready);
        lru_sync<2, kLruThreads>(group);
        F2 sum = both(0.f);
        if (plan.t.seq >= 0) {
            F2 state = me.fronts[warp][pair];
            if (second) state = fma2(decay, state, other);
#pragma unroll
            for (int j = 0; j < kLruRun; ++j) {
                const F2 after = fma2(a[j], state, h[j]);
                h[j] = state;                               // the state in front of the token
                state = after;
            }
            F2 e = fma2(me.behind[warp][pair].decay, me.carry[pair], me.behind[warp][pair].back);
            if (!second) e = fma2(decay, e, other);
            const int64_t tile = plan.t.first * p.D + plan.t.col * kLruCols;      // offsets within a tile have 32 bits
            IO *const xp = dx + tile, *const rp = dr + tile, *const ip = di + tile;
            F2 behind = both(1.f);                               // the decay of the token behind; sums that follow a product are
                                                                // written as one operation, or the loops below differ in it
            unsigned at = (unsigned)(row + kLruRun - 1) * (unsigned)p.D + pair * 2;
            const auto token = [&](int j, bool far, bool all) {
                e = fma2(e, behind, lru_read(from + 2 * N, row + j, pair));
                behind = a[j];
                const F2 shut = GATE ? aside.shut(j) : 0, g = GATE ? rcp_2(add2(shut, both(1.f))) : 0;
                const F2 x = lru_read(from + N, row + j, pair), eg = GATE ? mul2(e, g) : e, ea = mul2(e, a[j]);
                F2 dr_, s = part[j];
                if (RATE) {
                    const Parts o = parts_of(part[j], a[j], far);
                    s = o.s;
                    // -dlog a v = e a (a g x v / s - h v); dr is that times (1 - q) / 2
                    const F2 gxa = mul2(GATE ? mul2(g, x) : x, a[j]);
                    const F2 term = fma2(gxa, o.ratio, mul2(h[j], o.v)), base = mul2(ea, term);
                    sum = fma2(ea, term, sum);
                    dr_ = mul2(base, aside.half(j, row, pair));
                } else {
                    dr_ = mul2(mul2(a[j], s), fma2(e, h[j], neg2(mul2(eg, x))));
                }
                const F2 dx_ = mul2(eg, s);
                store2(xp + at, dx_, all ? 2 : left, all);
                store2(rp + at, dr_, all ? 2 : left, all);
                if (GATE) store2(ip + at, mul2(mul2(dx_, x), mul2(shut, g)), all ? 2 : left, all);
            };
            if (p.vec && len == kLruTile && left > 0 && !(RATE && plan.far)) {
#pragma unroll
                for (int j = kLruRun - 1; j >= 0; --j) {
                    token(j, false, true);
                    at -= (unsigned)p.D;
                }
            } else {
#pragma unroll
                for (int j = kLruRun - 1; j >= 0; --j) {
                    if (row + j < len) token(j, RATE && plan.far, false);
                    at -= (unsigned)p.D;
                }
            }
        }
        if (RATE) {
            sum = add2(sum, swap_halves(sum));
            if (!second) me.sums[warp][pair] = sum;
        }
        lru_sync<3, kLruWorkers>(group);                         // the tile has been read
        if (!TMA) fetch(turn + B);
        else if (thread == kLruWorkers - 32) issue(turn + B);
        if (RATE && warp == turn % kLruWarps && !second && plan.t.number != ~0u) {
            sum = me.sums[0][pair];
#pragma unroll
            for (int w = 1; w < kLruWarps; ++w) sum = add2(sum, me.sums[w][pair]);
            put_state2(dlam, (int64_t)plan.t.number * p.D + ch,
                       mul2(sum, *reinterpret_cast<const F2*>(plan.slopes + pair * 2)), left);
        }
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
    Lru p = lru_of(args, t, kGroups);
    p.vec = true;
    for (const void* v : {(const void*)g.dx, (const void*)g.dr, (const void*)g.di}) p.vec = p.vec && lru_pairs(v, args.D, es);
    const bool dy_vec = reinterpret_cast<uintptr_t>(g.dy) % 16 == 0 && args.D * es % 16 == 0;
    const LruRows dy = lru_rows(RowTensor{g.dy, args.D, dy_vec}, es);
    LruChain chain;
    if (cudaError_t e = lru_chain(args, t.lam, workspace, &chain, s)) return e;
    LruMaps m;
    const bool tma = args.total > 0 && p.x.unit == 16 && p.r.unit == 16 && dy.unit == 16 && (!p.i.p || p.i.unit == 16);
    if (tma && !(lru_map(&m.x, p.x, args) && lru_map(&m.r, p.r, args) && lru_map(&m.dy, dy, args) &&
                 (!p.i.p || lru_map(&m.i, p.i, args))))
        return cudaErrorInvalidValue;
    const cudaError_t e = lru_types(args.io, t.lam, t.i.p, [&](auto io, auto rate, auto gate) {
        using IO = decltype(io);
        constexpr bool R = decltype(rate)::value, G = decltype(gate)::value;
        const auto go = [&](auto kernel, int bytes) {
            return lru_launch(kernel, p, chain, kGroups * kLruThreads, kGroups * bytes, s, m, dy, kept,
                              g.dh_final, (IO*)g.dx, (IO*)g.dr, (IO*)g.di, partial, g.dh0);
        };
        return tma ? go(lru_backward_kernel<IO, R, G, true>, lru_backward_smem<IO, R, G, true>())
                   : go(lru_backward_kernel<IO, R, G, false>, lru_backward_smem<IO, R, G, false>());
    });
    if (e != cudaSuccess || !t.lam) return e;
    return column_sum(partial, lru_tiles(args), args.D, args.D, g.dlam, 0, nullptr, s);
}

}  // namespace layer
}  // namespace gdr
