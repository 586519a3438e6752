// What the forward, the gradient and the single-token form of the gated linear recurrence share.
//
//   h_t = a_t h_{t-1} + s_t g_t x_t,   q = sigmoid(r_t), g = sigmoid(i_t) (1 without i)
//   RATE:  a = e^{-k q}, k = c softplus(lam), s = sqrt(1 - a^2);     else  a = q, s = 1 - a
//
// A thread takes two neighbouring channels through the packed fp32 instructions.
#pragma once

#include <algorithm>
#include <type_traits>

#include "blackwell.cuh"
#include "gdr_internal.h"
#include "layer_common.cuh"
#include "layer_internal.h"
#include "tma_host.h"

namespace gdr {
namespace layer {

// A tile: 128 tokens of a sequence by 32 channels, a group's work: 16 runs of 8 tokens, each on 16 lanes of two channels.
// A block, one an SM, has as many groups as the registers hold, on neighbouring tiles of a strip of channels: a state goes
// from one group to the next through shared memory, and only the first group's comes from another block.
constexpr int kLruRun = 8, kLruRuns = 16, kLruTile = kLruRun * kLruRuns, kLruCols = 32, kLruPairs = kLruCols / 2;
constexpr int kLruWorkers = kLruRuns * kLruPairs, kLruWarps = kLruWorkers / 32;
constexpr int kLruThreads = kLruWorkers + 32;     // of a group: the workers and a warp that guides them
static_assert(kLruTile == kLruKept, "a kept state for each tile");

// A tensor of tokens, copied in aligned units of 16 bytes (by TMA), of 4, or (16-bit rows that start anywhere) by elements.
struct LruRows {
    const void* p;
    int64_t ld;
    int unit;
};

// Division of numbers below 2^31 by one that the host knows: q = x m >> 31 + l, m = ceil(2^(31 + l) / d), 2^l >= d.
struct Divisor {
    unsigned d = 1, m = 0, l = 0;
    __device__ __forceinline__ unsigned of(unsigned x) const { return d == 1 ? x : __umulhi(x, m) >> (l - 1); }
};
inline Divisor divisor(unsigned d) {
    Divisor v;
    v.d = d;
    while ((uint64_t{1} << v.l) < d) ++v.l;
    if (d > 1) v.m = (unsigned)(((uint64_t{1} << (31 + v.l)) + d - 1) / d);
    return v;
}

// The operator as the kernels take it.
struct Lru {
    Seqs q;
    int D;
    unsigned cols, tiles;    // strips of channels, and tiles of the token axis
    unsigned per;            // tiles of a sequence of a batch
    unsigned jobs;           // of the blocks: as many tiles of a strip as there are groups
    bool in_turns;           // the jobs of a batch's sequences take turns
    Divisor by_cols, by_n, by_per;
    LruRows x, r, i;
    const float *lam, *h0;
    float c;
    bool vec;                // outputs: two neighbouring channels are one aligned access
};

// ex2.approx leans low near 1 (see ssm.cuh): the exponent of a decay leans up by as much.
constexpr float kLruLean = 8e-9f;

__device__ __forceinline__ F2 neg2(F2 v) { return v ^ 0x8000000080000000ull; }

template <typename IO> __device__ __forceinline__ void store2(IO* p, F2 v, int left, bool vec) {
    const float2 f = unpack2(v);
    RawN<IO, 2> r;
    from_f2(r.e, f.x, f.y);
    if (vec && left >= 2) {
        if constexpr (sizeof(IO) == 4) *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(&r);
        else *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<const uint32_t*>(&r);
    } else {
        if (left > 0) p[0] = r.e[0];
        if (left > 1) p[1] = r.e[1];
    }
}
template <typename IO> __device__ __forceinline__ F2 wide2(const RawN<IO, 2>& r) {
    const float2 f = to_f2(r.e);
    return pack2(f.x, f.y);
}
// fp32 pairs of [.., D] that start anywhere; zeros without p or past the row.
__device__ __forceinline__ F2 state2(const float* p, int64_t at, int left) {
    return pack2(p && left > 0 ? p[at] : 0.f, p && left > 1 ? p[at + 1] : 0.f);
}
__device__ __forceinline__ void put_state2(float* p, int64_t at, F2 v, int left) {
    const float2 f = unpack2(v);
    if (left > 0) p[at] = f.x;
    if (left > 1) p[at + 1] = f.y;
}

__device__ __forceinline__ float min_nan(float a, float b) {   // NaN where either is
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float sqrt_fast(float x) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ F2 sqrt2(F2 v) {
    const float2 f = unpack2(v);
    return pack2(sqrt_fast(f.x), sqrt_fast(f.y));
}
// A channel's k = c softplus(lam), and its slope c sigmoid(lam).
__device__ __forceinline__ float rate_of(float lam, float c) {
    return c * (fmaxf(lam, 0.f) + log1pf(expf(-fabsf(lam))));     // a NaN comes through the logarithm
}
// k, sqrt(2 k), and k's slope by lam over 2 k, which is zero for a channel that neither forgets nor takes.
__device__ __forceinline__ float4 rates_of(float lam, float c) {
    const float k = rate_of(lam, c), slope = c / (1.f + expf(-lam));
    return make_float4(k, sqrtf(2.f * k), k > 1e-37f ? slope / (2.f * k) : 0.f, 0.f);
}

// Of each channel `yes` where x is below, above the bound, else (or NaN) `no`.
__device__ __forceinline__ F2 below(F2 x, float bound, F2 yes, F2 no) {
    const float2 at = unpack2(x), y = unpack2(yes), n = unpack2(no);
    return pack2(at.x < bound ? y.x : n.x, at.y < bound ? y.y : n.y);
}
__device__ __forceinline__ F2 above(F2 x, float bound, F2 yes, F2 no) {
    const float2 at = unpack2(x), y = unpack2(yes), n = unpack2(no);
    return pack2(at.x > bound ? y.x : n.x, at.y > bound ? y.y : n.y);
}
// A token's decay a and input's part s; q = sigmoid(r).
//
// RATE: s^2 = 1 - e^-v with v = 2 k q: by a polynomial where 1 - a^2 cancels.  Else the smaller of a and s comes from e^-|r| to
// relative accuracy, and the other is 1 less it, which is exact where a state is kept.
template <bool RATE> __device__ __forceinline__ void decay_and_part(F2 r, F2 k, F2& a, F2& s, F2& q) {
    if (RATE) {
        q = sigmoid2(r);
        const F2 kq = mul2(k, q), v = add2(kq, kq);
        a = ex2_2(fma2(kq, both(-kLog2e), both(kLruLean)));
        // (1 - e^-v) / v up to v = 1/2, the best polynomial of degree 4: off by 1.1e-7
        F2 m = fma2(v, both(0x1.bb955ap-8f), both(-0x1.4fdc9cp-5f));
        m = fma2(v, m, both(0x1.5516c6p-3f));
        m = fma2(v, m, both(-0x1.fffe02p-2f));
        m = mul2(v, fma2(v, m, both(0x1.fffffep-1f)));
        const float2 near = unpack2(m), far = unpack2(fma2(mul2(a, both(-1.f)), a, both(1.f))), at = unpack2(v);
        s = sqrt2(pack2(at.x < 0.5f ? near.x : far.x, at.y < 0.5f ? near.y : far.y));
    } else {
        const float2 f = unpack2(r);
        const F2 e = pack2(ex2(-fabsf(f.x) * kLog2e), ex2(-fabsf(f.y) * kLog2e));
        const F2 small = mul2(e, rcp_2(add2(e, both(1.f)))), rest = fma2(small, both(-1.f), both(1.f));
        a = below(r, 0.f, small, rest);
        s = below(r, 0.f, rest, small);
        q = a;
    }
}

// The same for a whole run at fewer reciprocals and roots, which take twice the time of 2^x and four times that of a product
// (an SM does 16 of them a clock; formed one by one they bound the forward with rates at 134 of 158 us for 32768 x 4096).
//
// RATE, where v = 2 k q stays below 1/2 (k <= 1/4: gates that keep more than 0.78 of a state when they are open): with
// w = sqrt(q) = (1 + e^-r)^-1/2, s = sqrt(2 k) w P(v), P(v) = sqrt((1 - e^-v) / v), by a polynomial; one root of
// (1 + e^-r)(1 + e^-i)^2 gives w g, times (1 + e^-i) it gives w.  The product must not overflow where g is small: i is at least
// -27.  A gate r so far shut that it still does (an inflow below 2^-64 of x) lets nothing in.
// Else: q = 1 / (1 + e^-r), s = e^-r q, and a = 1 - s, exact where a state is kept but off by up to 4e-7: below r = -3 a is q.
// (q near 1 is rounded once a token, which a long life adds up; from -3 on the 4e-7 are below 1e-5 of a.)
//
// A warp goes by these alone where every token and channel of its runs may; elsewhere it forms the others' terms too and
// selects, so that a token's bits follow from its own channel's numbers, whatever its neighbours hold.  What that costs (8192 x
// 4096 bf16, forward and gradient): all k <= 1/4 62 and 120 us, k up to 0.84 or to 5 71 and 156.
constexpr float kLruSlow = 0.25f, kLruNear = 0.50001f;      // the largest k, and what v stays below when q is rounded up
constexpr float kLruLeast = -27.f, kLruJoint = 0x1p39f;     // the least i, and what 1 + e^27 stays below
constexpr float kLruShut = -3.f, kLruShutE = 20.086f;       // the least r that has a = 1 - s, and what e^3 stays below
constexpr float kLruHuge = 0x1.8p126f;      // what an infinite e^-r or e^-i is cut to: 1 / (1 + it) is still flushed to zero
__device__ __forceinline__ float rsqrt_fast(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ F2 rsqrt2(F2 v) {
    const float2 f = unpack2(v);
    return pack2(rsqrt_fast(f.x), rsqrt_fast(f.y));
}
__device__ __forceinline__ F2 one_and_exp(F2 v) { return add2(ex2_2(mul2(v, both(-kLog2e))), both(1.f)); }    // 1 + e^-v
__device__ __forceinline__ F2 lru_p(F2 v) {      // off by 9e-9 up to 1/2
    F2 p = fma2(v, both(0x1.9419eap-11f), both(-0x1.fd8e2ep-8f));
    p = fma2(v, p, both(0x1.aa9cb4p-5f));
    p = fma2(v, p, both(-0x1.ffffc8p-3f));
    return fma2(v, p, both(1.f));
}
__device__ __forceinline__ F2 lru_p_inverse(F2 v) {      // 1 / P(v), off by 4e-8
    F2 p = fma2(v, both(-0x1.5d5098p-9f), both(0x1.55d41ap-7f));
    p = fma2(v, p, both(0x1.ffff5p-3f));
    return fma2(v, p, both(1.f));
}
// RATE: w and z = w g from t1 = 1 + e^-r and t2 = 1 + e^-i.  WILD: i may be anything.
template <bool GATE, bool WILD> __device__ __forceinline__ void lru_roots(F2 t1, F2 t2, F2& w, F2& z) {
    if (GATE) {
        z = rsqrt2(mul2(t1, mul2(t2, t2)));
        w = mul2(z, t2);
        if (WILD) {
            const F2 alone = rsqrt2(t1);
            z = below(t2, kLruJoint, z, mul2(alone, rcp_2(t2)));
            w = below(t2, kLruJoint, w, alone);
        }
    } else {
        z = w = rsqrt2(t1);
    }
}
// Else: a, its complement s, and s g; t2 = 1 + e^-i.  SHUT: r may be below kLruShut.
template <bool GATE, bool SHUT> __device__ __forceinline__ void lru_parts(F2 r, F2 t2, F2& a, F2& s, F2& sg) {
    const F2 e = ex2_2(mul2(r, both(-kLog2e))), q = rcp_2(add2(e, both(1.f)));
    s = mul2(e, q);
    a = fma2(s, both(-1.f), both(1.f));
    if (SHUT) {
        a = below(e, kLruShutE, a, q);
        s = above(e, 0x1p100f, both(1.f), s);           // q is flushed to zero from 2^126 on
    }
    sg = GATE ? mul2(s, rcp_2(t2)) : s;
}

// Minima of two channels, NaN where either is.
__device__ __forceinline__ RawN<float, 2> min_pair(RawN<float, 2> a, RawN<float, 2> b) {
    return {min_nan(a.e[0], b.e[0]), min_nan(a.e[1], b.e[1])};
}
template <typename IO> __device__ __forceinline__ RawN<IO, 2> min_pair(RawN<IO, 2> a, RawN<IO, 2> b) {
    using Two = std::conditional_t<std::is_same_v<IO, __half>, __half2, __nv_bfloat162>;
    RawN<IO, 2> r;
    *reinterpret_cast<Two*>(&r) = __hmin2_nan(*reinterpret_cast<const Two*>(&a), *reinterpret_cast<const Two*>(&b));
    return r;
}
// ---------------------------------------------------------------- tiles and their order

struct LruTile {
    int seq;                 // -1: no such tile
    unsigned number, col;    // of the tile over all sequences, of its channels
    int64_t first;           // its first token on the axis
    int len;                 // tokens, 0 of an empty sequence
    unsigned to_head, to_tail;  // tiles before it and behind it in its sequence
};

// Group `group`'s tile of a job.  Jobs go through all strips before they go on in time, each after those it waits for (BACK:
// from behind); where there are few strips the sequences of a batch take turns, so that a job's neighbour in time is long
// done.  A job's last tiles may not exist (`number` is ~0 then).
template <bool BACK, int GROUPS> __device__ __forceinline__ LruTile lru_tile(const Lru& a, unsigned job, unsigned group) {
    LruTile t;
    const unsigned row = a.by_cols.of(job);
    t.col = job - row * a.cols;
    int64_t len = 0;
    unsigned tile = 0;
    bool some;
    if (a.in_turns) {
        const unsigned k = a.by_n.of(row);
        t.seq = (int)(row - k * (unsigned)a.q.n);
        tile = k * GROUPS + group;
        some = tile < a.per;
        if (BACK) tile = a.per - 1 - tile;
        t.number = (unsigned)t.seq * a.per + tile;
    } else {
        t.number = row * GROUPS + group;
        some = t.number < a.tiles;
        if (BACK) t.number = a.tiles - 1 - t.number;
        if (!a.q.cu) {
            t.seq = (int)a.by_per.of(some ? t.number : 0);
            tile = t.number - (unsigned)t.seq * a.per;
        }
    }
    t.first = 0;
    if (some && a.q.cu) {
        const TileAt at = find_tile(a.q, t.number, kLruTile);
        t.seq = at.seq;
        t.first = at.start;
        len = at.len;
        tile = (unsigned)at.tile;
    } else if (some) {
        t.first = t.seq * a.q.T;
        len = a.q.T;
    }
    if (!some) t.seq = -1, t.number = ~0u;
    t.first += (int64_t)tile * kLruTile;
    len -= (int64_t)tile * kLruTile;
    t.len = t.seq < 0 ? 0 : (int)(len < kLruTile ? len : kLruTile);
    t.to_head = t.seq < 0 ? 0 : tile;
    t.to_tail = t.seq < 0 || len <= kLruTile ? 0 : (unsigned)((len - 1) / kLruTile);
    return t;
}

// What the blocks of a launch tell one another.  Everything starts as 0xff bytes: a NaN that no arithmetic makes says that a
// word is not written yet.  Each word is written once, whole, so it needs no flag and no fence.
struct LruChain {
    ulonglong2* maps;        // [tiles][cols][pairs]: a tile makes of state h  h * x + y; nullptr: no tile waits for another
    F2* states;              // [tiles][cols][pairs]: the state that a tile goes on from
    const float4* rates;     // [cols * 32]: rates_of each channel, or nullptr (the guides form them)
    unsigned* err;           // the device error word
};
inline size_t lru_chain_bytes(int64_t tiles, int64_t cols) {       // the maps, the states, the rates
    return (size_t)tiles * cols * kLruPairs * 24 + (size_t)cols * kLruCols * 16;
}

__device__ __forceinline__ F2 written(F2 v) {         // a payload that says "not written" becomes the usual NaN
    return (uint32_t)v == 0xffffffffu ? (v & 0xffffffff00000000ull) | 0x7fffffffu : v;
}
__device__ __forceinline__ bool is_written(F2 v) { return (uint32_t)v != 0xffffffffu; }
__device__ __forceinline__ void publish_map(ulonglong2* p, F2 decay, F2 own) {
    asm volatile("st.relaxed.gpu.global.v2.u64 [%0], {%1, %2};" ::"l"(p), "l"(written(decay)), "l"(written(own)) : "memory");
}
__device__ __forceinline__ void publish_state(F2* p, F2 v) {
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(written(v)) : "memory");
}
__device__ __forceinline__ ulonglong2 look_map(const ulonglong2* p) {
    ulonglong2 v;
    asm volatile("ld.relaxed.gpu.global.v2.u64 {%0, %1}, [%2];" : "=l"(v.x), "=l"(v.y) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ F2 look_state(const F2* p) {
    F2 v;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}

constexpr int kLruLook = 4;

// One look for the state that tile `t` goes on from, for the warp's channel pair at `pair`: the nearest one written among its
// own and those of the kLruLook - 1 tiles before it (`near` of them in its sequence), taken through the maps of the tiles
// between.  These are applied one by one, from the state on, as the tiles themselves do: wherever the state comes from, the
// bits are the same.  BACK: the tiles that come before are those behind.
template <bool BACK>
__device__ __forceinline__ bool look_back(const LruChain& c, const LruTile& t, unsigned cols, int pair, unsigned near,
                                          F2& state) {
    const int64_t at = ((int64_t)t.number * cols + t.col) * kLruPairs + pair;
    const int64_t step = (BACK ? 1 : -1) * (int64_t)cols * kLruPairs;
    F2 s[kLruLook];
    ulonglong2 m[kLruLook];
#pragma unroll
    for (int j = 0; j < kLruLook; ++j) {           // s[j]: the state j tiles before; m[j]: the map of the tile after it
        s[j] = ~0ull;
        m[j] = make_ulonglong2(~0ull, ~0ull);
        if ((unsigned)j < near) s[j] = look_state(c.states + at + j * step);
        if ((unsigned)j + 1 < near && j + 1 < kLruLook) m[j] = look_map(c.maps + at + (j + 1) * step);
    }
    bool found = false, linked = true;
    int from = 0;
#pragma unroll
    for (int j = 0; j < kLruLook; ++j) {
        if (!found && linked && is_written(s[j])) found = true, state = s[j], from = j;
        linked = linked && is_written(m[j].x) && is_written(m[j].y);
    }
    if (!__all_sync(0xffffffffu, found)) return false;
#pragma unroll
    for (int j = kLruLook - 2; j >= 0; --j)
        if (j < from) state = fma2(m[j].x, state, m[j].y);
    return true;
}
// The same until it is found.  A wait that runs out (about a second) sets the error word and goes on with zeros.
constexpr int kLruPolls = 1 << 20;
template <bool BACK>
__device__ __forceinline__ F2 wait_back(const LruChain& c, const LruTile& t, unsigned cols, int pair, unsigned near) {
    F2 state = 0;
    for (int poll = 0; poll < kLruPolls; ++poll) {
        if (look_back<BACK>(c, t, cols, pair, near, state)) return state;
        if ((poll & 4095) == 4095 && *reinterpret_cast<volatile unsigned*>(c.err)) break;
    }
    if ((threadIdx.x & 31) == 0) atomicCAS(c.err, 0u, kDeviceErrTimeout);
    return 0;
}

// Named barriers of a group: 1 and 3 of the workers, 2 of all, where the guide only arrives.  Their names are known to the
// compiler: from registers they take several times as long.
template <int ID, int N> __device__ __forceinline__ void lru_sync(int group) {
    if (group == 0) asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(N) : "memory");
    else if (group == 1) asm volatile("bar.sync %0, %1;" ::"n"(ID + 3), "n"(N) : "memory");
    else asm volatile("bar.sync %0, %1;" ::"n"(ID + 6), "n"(N) : "memory");
}
template <int ID, int N> __device__ __forceinline__ void lru_arrive(int group) {
    if (group == 0) asm volatile("bar.arrive %0, %1;" ::"n"(ID), "n"(N) : "memory");
    else if (group == 1) asm volatile("bar.arrive %0, %1;" ::"n"(ID + 3), "n"(N) : "memory");
    else asm volatile("bar.arrive %0, %1;" ::"n"(ID + 6), "n"(N) : "memory");
}
__device__ __forceinline__ F2 swap_halves(F2 v) { return __shfl_xor_sync(0xffffffffu, v, 16); }

// What the guide tells the workers of a tile; rates alone have a `far`.
constexpr int kLruPlans = 4;
struct LruPlan {
    LruTile t;
    bool live;               // there is one
    bool far;                // some channel's rate is above kLruSlow
    alignas(8) float rates[kLruCols], roots[kLruCols], slopes[kLruCols];       // rates_of
};
// The guide's: a channel's rates are read four tiles ahead and a tile planned three ahead, after the present one's state is
// out, so that no way to memory holds anyone up.
template <bool BACK, bool RATE, int GROUPS> struct LruPlanner {
    float4 rate;             // of the tile to be planned: rates_of

    __device__ __forceinline__ unsigned job(unsigned turn) const { return blockIdx.x + turn * gridDim.x; }
    __device__ __forceinline__ void read(const Lru& p, const LruChain& c, unsigned turn) {
        if (!RATE || job(turn) >= p.jobs) return;
        const unsigned col = job(turn) - p.by_cols.of(job(turn)) * p.cols;
        const int ch = (int)col * kLruCols + (threadIdx.x & 31);
        if (c.rates) rate = c.rates[ch];
        else rate = ch < p.D ? rates_of(p.lam[ch], p.c) : float4{};
    }
    // Plans the tile of turn `turn`, in order.
    __device__ __forceinline__ void plan(const Lru& p, const LruChain& c, unsigned turn, unsigned group, LruPlan* plan) {
        const int lane = threadIdx.x & 31;
        const bool live = job(turn) < p.jobs;
        if (lane == 0) plan->live = live;
        if (live) {
            const LruTile t = lru_tile<BACK, GROUPS>(p, job(turn), group);
            if (lane == 0) plan->t = t;
            if (RATE) {
                const bool far = __any_sync(0xffffffffu, rate.x > kLruSlow);
                if (lane == 0) plan->far = far;
                plan->rates[lane] = rate.x;
                plan->roots[lane] = rate.y;
                if (BACK) plan->slopes[lane] = rate.z;
            }
        }
        read(p, c, turn + 1);
        __syncwarp();
    }
};

// The way of a state from a group to the next one: given once a turn, and taken before it is given again.
struct LruHand {
    F2 state[kLruPairs];
    uint64_t given, taken;
};
__device__ __forceinline__ void lru_give(LruHand& h, F2 state, unsigned turn, unsigned* err) {      // by a warp
    if (turn > 0) bw::mbar_wait(&h.taken, turn - 1 & 1, err, kDeviceErrTimeout);
    if ((threadIdx.x & 31) < kLruPairs) h.state[threadIdx.x & 31] = state;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) bw::mbar_arrive(&h.given);
}
__device__ __forceinline__ F2 lru_take(LruHand& h, unsigned turn, unsigned* err) {
    bw::mbar_wait(&h.given, turn & 1, err, kDeviceErrTimeout);
    const F2 state = h.state[threadIdx.x % kLruPairs];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) bw::mbar_arrive(&h.taken);
    return state;
}

// Inputs on their way by TMA: a box of a tile's rows and 32 channels, zeros outside the tensor.  (Boxes of the rows that the
// short sequences of a batch have save nothing: 2000 x 16 x 4096 803 us with them, 799 without; gradient 3,458 and 3,460.)
struct LruMaps {
    CUtensorMap r, x, i, dy;
};
// One lane's request for a tile of a tensor.
template <typename IO>
__device__ __forceinline__ void lru_tma(IO* to, const CUtensorMap* map, uint64_t* bar, const LruTile& t) {
    bw::tma_load_4d(to, map, bar, (int)t.col * kLruCols * (int)sizeof(IO) / 2, (int)t.first, 0, 0);
}

// ---------------------------------------------------------------- inputs

// Without TMA the workers copy: rows on 16-byte boundaries in such units, others in units of 4 bytes or by elements.
template <int UNIT> __device__ __forceinline__ void lru_copy(void* to, const void* from, int bytes) {
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
    if (UNIT == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(from), "r"(bytes) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(at), "l"(from), "r"(bytes) : "memory");
}
template <typename IO, int UNIT>
__device__ __forceinline__ void lru_fetch_units(const LruRows& v, const LruTile& t, int D, int thread, IO* to) {
    constexpr int per = UNIT / (int)sizeof(IO), pieces = kLruCols / per, step = kLruWorkers / pieces;
    const int piece = thread % pieces, ch = t.col * kLruCols + piece * per;
    const int bytes = min(per, D - ch) * (int)sizeof(IO);
    if (bytes <= 0) return;
    const IO* from = (const IO*)v.p + (t.first + thread / pieces) * v.ld + ch;
#pragma unroll
    for (int k = 0; k < kLruTile / step; ++k) {
        const int row = thread / pieces + k * step;
        if (row < t.len) lru_copy<UNIT>(to + row * kLruCols + piece * per, from, bytes);
        from += step * v.ld;
    }
}
// A tile of a tensor on its way into shared memory, by the workers; rows past the tile's end stay what they were.
template <typename IO>
__device__ __forceinline__ void lru_fetch(const LruRows& v, const LruTile& t, int D, int thread, IO* to) {
    if (v.unit == 16) {
        lru_fetch_units<IO, 16>(v, t, D, thread, to);
    } else if (sizeof(IO) == 4 || v.unit >= 4) {
        lru_fetch_units<IO, 4>(v, t, D, thread, to);
    } else {
        constexpr int step = kLruWorkers / kLruPairs, most = kLruTile / step;
        const int piece = thread % kLruPairs, ch = t.col * kLruCols + piece * 2, row0 = thread / kLruPairs;
        const IO* from = (const IO*)v.p + (t.first + row0) * v.ld + ch;
        RawN<IO, 2> e[most];
#pragma unroll
        for (int k = 0; k < most; ++k) {
            const bool live = row0 + k * step < t.len;
            e[k].e[0] = live && ch < D ? from[0] : from_f<IO>(0.f);
            e[k].e[1] = live && ch + 1 < D ? from[1] : from_f<IO>(0.f);
            from += step * v.ld;
        }
#pragma unroll
        for (int k = 0; k < most; ++k)
            *reinterpret_cast<RawN<IO, 2>*>(to + (row0 + k * step) * kLruCols + piece * 2) = e[k];
    }
}

// A token of the thread's run, two channels; past the tile's end anything.
template <typename IO> __device__ __forceinline__ RawN<IO, 2> lru_raw(const IO* from, int row, int pair) {
    return *reinterpret_cast<const RawN<IO, 2>*>(from + row * kLruCols + pair * 2);
}
template <typename IO> __device__ __forceinline__ F2 lru_read(const IO* from, int row, int pair) {
    return wide2(lru_raw(from, row, pair));
}
// Whether a run's gates are all at least `bound`, and none NaN; tokens past the tile's end and channels past the last, which
// hold anything, are not asked.
template <typename IO>
__device__ __forceinline__ bool lru_above(const RawN<IO, 2> (&v)[kLruRun], float bound, int live, int left) {
    RawN<IO, 2> least = v[0];
    if (live >= kLruRun) {
#pragma unroll
        for (int j = 1; j < kLruRun; ++j) least = min_pair(least, v[j]);
    } else {
#pragma unroll
        for (int j = 1; j < kLruRun; ++j)
            if (j < live) least = min_pair(least, v[j]);
    }
    const float2 g = to_f2(least.e);
    return live <= 0 || ((left < 1 || g.x >= bound) && (left < 2 || g.y >= bound));
}
// Whether no gate of the warp's runs is so far shut that the short formulas are not enough.  GATE: whether i is asked.
template <bool RATE, bool GATE, typename IO>
__device__ __forceinline__ bool lru_tame(const RawN<IO, 2> (&r)[kLruRun], const RawN<IO, 2> (&i)[kLruRun], int live, int left) {
    bool ok = true;
    if (!RATE) ok = lru_above(r, kLruShut, live, left);
    if (GATE) ok = ok && lru_above(i, kLruLeast, live, left);
    return (RATE && !GATE) || __all_sync(0xffffffffu, ok);
}

// Calls f with a value of the io type and whether there are rates and input gates.
template <typename F> cudaError_t lru_types(int io, bool rate, bool gate, F f) {
    const auto forms = [&](auto v) {
        if (rate) return gate ? f(v, std::true_type(), std::true_type()) : f(v, std::true_type(), std::false_type());
        return gate ? f(v, std::false_type(), std::true_type()) : f(v, std::false_type(), std::false_type());
    };
    if (io == GDR_F32) return forms(float());
    if (io == GDR_BF16) return forms(__nv_bfloat16());
    return forms(__half());
}

inline bool lru_pairs(const void* p, int64_t ld, int64_t e) {
    return reinterpret_cast<uintptr_t>(p) % (2 * e) == 0 && ld % 2 == 0;
}
inline LruRows lru_rows(const RowTensor& t, int64_t e) {
    const bool four = reinterpret_cast<uintptr_t>(t.p) % 4 == 0 && t.ld * e % 4 == 0;
    return LruRows{t.p, t.ld, t.vec ? 16 : four ? 4 : 2};
}
inline Lru lru_of(const LruArgs& a, const LruTensors& t, int groups) {
    const int64_t e = a.io == GDR_F32 ? 4 : 2;
    Lru k{};
    k.q = Seqs{a.cu, a.total, a.T, (int)a.n};
    k.D = a.D;
    k.cols = (unsigned)((a.D + kLruCols - 1) / kLruCols);
    k.tiles = (unsigned)lru_tiles(a);
    k.per = k.tiles / (unsigned)a.n;
    k.by_cols = divisor(k.cols);
    k.by_n = divisor((unsigned)a.n);
    k.by_per = divisor(k.per ? k.per : 1);
    // in turns at the price of the last job's idle groups; a strip has about 152 / cols jobs in flight
    k.in_turns = !a.cu && a.n > 1 && k.cols < 64 && k.per >= 4 * (unsigned)groups;
    k.jobs = k.cols * (k.in_turns ? (k.per + groups - 1) / groups * (unsigned)a.n : (k.tiles + groups - 1) / groups);
    k.x = lru_rows(t.x, e);
    k.r = lru_rows(t.r, e);
    k.i = lru_rows(t.i, e);
    k.lam = t.lam;
    k.h0 = t.h0;
    k.c = a.c;
    return k;
}

inline bool lru_map(CUtensorMap* m, const LruRows& v, const LruArgs& a) {
    const uint64_t e = a.io == GDR_F32 ? 4 : 2, ld = (uint64_t)v.ld * e, rows = (uint64_t)a.total;
    const uint64_t dims[4] = {(uint64_t)a.D * e / 2, rows, 1, 1}, strides[3] = {ld, ld, ld};
    const uint32_t box[4] = {kLruCols * (uint32_t)e / 2, kLruTile, 1, 1};
    return make_tmap_bf16_4d_mode(m, v.p, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);   // copies any type's bits
}

inline bool lru_one_tile_each(const LruArgs& a) { return (a.cu ? a.total : a.T) <= kLruTile; }
// One block an SM at most, of those that the context has; blocks that wait for one another run together or not at all.
template <typename... A, typename... B>
cudaError_t lru_launch(void (*kernel)(A...), const Lru& p, const LruChain& c, int threads, int bytes, cudaStream_t s,
                       B... args) {
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) return e;
    int device = 0, sms = 0;
    if (cudaError_t e = cudaGetDevice(&device)) return e;
    if (cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device)) return e;
    cudaLaunchAttribute together{};
    together.id = cudaLaunchAttributeCooperative;
    together.val.cooperative = 1;
    cudaLaunchConfig_t config{};
    config.gridDim = dim3(std::min(p.jobs, (unsigned)sms));
    config.blockDim = dim3((unsigned)threads);
    config.dynamicSmemBytes = (size_t)bytes;
    config.stream = s;
    config.attrs = &together;
    config.numAttrs = c.maps ? 1 : 0;
    return cudaLaunchKernelEx(&config, kernel, p, c, args...);
}

// The chain's words in the workspace, made "not written", and the rates; none of them with one tile a sequence.
cudaError_t lru_chain(const LruArgs& a, const float* lam, void* workspace, LruChain* c, cudaStream_t s);

}  // namespace layer
}  // namespace gdr
