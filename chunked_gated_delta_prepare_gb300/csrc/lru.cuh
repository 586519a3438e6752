// What the forward, the gradient and the single-token form of the gated linear recurrence share.
//
//   h_t = a_t h_{t-1} + s_t g_t x_t,   q = sigmoid(r_t), g = sigmoid(i_t) (1 without i)
//   RATE:  a = e^{-k q}, k = c softplus(lam), s = sqrt(1 - a^2);     else  a = q, s = 1 - a
//
// A thread takes two neighbouring channels through the packed fp32 instructions.
#pragma once

#include <algorithm>
#include <type_traits>

#include "gdr_internal.h"
#include "layer_common.cuh"
#include "layer_internal.h"

namespace gdr {
namespace layer {

// A tile: 128 tokens of a sequence by 32 channels, a block's work: 16 runs of 8 tokens, each on 16 lanes of two channels.
// Narrow tiles leave few tiles of a strip of channels in flight at once, so a tile's state is never far away.
constexpr int kLruRun = 8, kLruRuns = 16, kLruTile = kLruRun * kLruRuns, kLruCols = 32, kLruPairs = kLruCols / 2;
constexpr int kLruWorkers = kLruRuns * kLruPairs, kLruThreads = kLruWorkers + 32;     // and a warp that guides them
static_assert(kLruTile == kLruKept, "a kept state for each tile");

// A tensor of tokens, copied in aligned units of 16 bytes, of 4, or (16-bit rows that start anywhere) by elements.
struct LruRows {
    const void* p;
    int64_t ld;
    int unit;
};

// The operator as the kernels take it.
struct Lru {
    Seqs q;
    int D;
    unsigned cols, tiles;    // blocks of channels, and tiles of the token axis
    LruRows x, r, i;
    const float *lam, *h0;
    float c;
    bool vec;                // outputs: two neighbouring channels are one aligned access
};

// ex2.approx leans low near 1 (see ssm.cuh): the exponent of a decay leans up by as much.
constexpr float kLruLean = 8e-9f;

__device__ __forceinline__ F2 neg2(F2 v) { return v ^ 0x8000000080000000ull; }

template <typename IO> __device__ __forceinline__ RawN<IO, 2> load2(const IO* p, int left, bool vec) {
    RawN<IO, 2> r;
    if (vec && left >= 2) {
        if constexpr (sizeof(IO) == 4) *reinterpret_cast<uint2*>(&r) = __ldg(reinterpret_cast<const uint2*>(p));
        else *reinterpret_cast<uint32_t*>(&r) = __ldg(reinterpret_cast<const uint32_t*>(p));
    } else {
        r.e[0] = left > 0 ? p[0] : from_f<IO>(0.f);
        r.e[1] = left > 1 ? p[1] : from_f<IO>(0.f);
    }
    return r;
}
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

// sigmoid(v) and 1 - sigmoid(v), both to relative accuracy: with e = e^-|v| <= 1 the smaller is e / (1 + e), the larger
// one less that.
__device__ __forceinline__ void sigmoid_both2(F2 v, F2& up, F2& down) {
    const float2 f = unpack2(v);
    const F2 e = pack2(ex2(-fabsf(f.x) * kLog2e), ex2(-fabsf(f.y) * kLog2e));
    const F2 small = mul2(e, rcp_2(add2(both(1.f), e))), large = fma2(small, both(-1.f), both(1.f));
    const float2 s = unpack2(small), l = unpack2(large);
    up = pack2(f.x < 0.f ? s.x : l.x, f.y < 0.f ? s.y : l.y);
    down = pack2(f.x < 0.f ? l.x : s.x, f.y < 0.f ? l.y : s.y);
}

// 1 - e^-v for v >= 0, given e^(-v/2) = a: 1 - a^2, and near 0, where that cancels, v (1 - v/2 + v^2/6 - ...), whose terms
// after v^4/120 are below 2^-24 of the sum at v = 1/8.
__device__ __forceinline__ F2 one_less(F2 v, F2 a) {
    F2 p = fma2(v, both(1.f / 120), both(-1.f / 24));
    p = fma2(v, p, both(1.f / 6));
    p = fma2(v, p, both(-1.f / 2));
    p = fma2(v, p, both(1.f));
    const float2 near = unpack2(mul2(v, p)), far = unpack2(fma2(mul2(a, both(-1.f)), a, both(1.f))), at = unpack2(v);
    return pack2(at.x < 0.125f ? near.x : far.x, at.y < 0.125f ? near.y : far.y);
}

__device__ __forceinline__ float rsqrt_fast(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / sqrt(v): finite for 0, and NaN is left to what it multiplies.
__device__ __forceinline__ F2 rsqrt2(F2 v) {
    const float2 f = unpack2(v);
    return pack2(rsqrt_fast(fmaxf(f.x, 1e-37f)), rsqrt_fast(fmaxf(f.y, 1e-37f)));
}
__device__ __forceinline__ F2 rcp2_finite(F2 v) {
    const float2 f = unpack2(v);
    return pack2(rcp(fmaxf(f.x, 3e-19f)), rcp(fmaxf(f.y, 3e-19f)));
}

// A channel's k = c softplus(lam), and its slope c sigmoid(lam).
__device__ __forceinline__ float rate_of(float lam, float c) {
    return c * (fmaxf(lam, 0.f) + log1pf(expf(-fabsf(lam))));     // a NaN comes through the logarithm
}
__device__ __forceinline__ float rate_slope(float lam, float c) { return c / (1.f + expf(-lam)); }

// A token's decay a and input's part s; q = sigmoid(r).
template <bool RATE> __device__ __forceinline__ void decay_and_part(F2 r, F2 k, F2& a, F2& s, F2& q) {
    if (RATE) {
        q = sigmoid2(r);
        const F2 kq = mul2(k, q);
        a = ex2_2(fma2(kq, both(-kLog2e), both(kLruLean)));
        const F2 m = one_less(add2(kq, kq), a);
        s = mul2(m, rsqrt2(m));
    } else {
        sigmoid_both2(r, a, s);
        q = a;
    }
}

// ---------------------------------------------------------------- tiles and their order

struct LruTile {
    int seq;                 // -1: no such tile
    unsigned number, col;    // of the tile over all sequences, of its channels
    int64_t first;           // its first token on the axis
    int len;                 // tokens, 0 of an empty sequence
    unsigned to_head, to_tail;  // tiles before it and behind it in its sequence
};

// Tiles in the order they are worked on: all channels of one after all of another, each after those it waits for (BACK: the
// tiles behind it).  The sequences of a batch take turns, so that a tile's neighbour in time is long done.
template <bool BACK> __device__ __forceinline__ LruTile lru_tile(const Lru& a, unsigned ticket) {
    LruTile t;
    unsigned k = ticket / a.cols;
    t.col = ticket - k * a.cols;
    if (BACK) k = a.tiles - 1 - k;
    int64_t len;
    unsigned tile;
    if (a.q.cu) {
        const TileAt at = find_tile(a.q, k, kLruTile);
        t.seq = at.seq;
        t.number = k;
        t.first = at.start;
        len = at.len;
        tile = (unsigned)at.tile;
    } else {
        tile = k / (unsigned)a.q.n;
        t.seq = (int)(k - tile * (unsigned)a.q.n);
        t.number = (unsigned)t.seq * (a.tiles / (unsigned)a.q.n) + tile;
        t.first = t.seq * a.q.T;
        len = a.q.T;
    }
    t.first += (int64_t)tile * kLruTile;
    len -= (int64_t)tile * kLruTile;
    t.len = t.seq < 0 ? 0 : (int)(len < kLruTile ? len : kLruTile);
    t.to_head = tile;
    t.to_tail = len <= kLruTile ? 0 : (unsigned)((len - 1) / kLruTile);
    return t;
}

// What the blocks of a launch tell one another.  Everything starts as 0xff bytes: a NaN that no arithmetic makes says that a
// word is not written yet.  Each word is written once, whole, so it needs no flag and no fence.
struct LruChain {
    unsigned* ticket;        // tiles taken so far, less one; nullptr: no tile waits for another
    ulonglong2* maps;        // [tiles][cols][pairs]: a tile makes of state h  h * x + y
    F2* states;              // [tiles][cols][pairs]: the state that a tile goes on from
    unsigned* err;           // the device error word
};
inline size_t lru_chain_bytes(int64_t tiles, int64_t cols) { return 256 + (size_t)tiles * cols * kLruPairs * 24; }

// A block's k-th tile.  Tiles are handed out in order, so those that a tile waits for belong to blocks that run already.
__device__ __forceinline__ unsigned take_ticket(const LruChain& c, unsigned k) {
    return c.ticket ? atomicAdd(c.ticket, 1u) + 1u : blockIdx.x + k * gridDim.x;
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

constexpr int kLruLook = 4, kLruPolls = 1 << 20;       // about a second

// The state that tile `t` goes on from, for the warp's channel pair at `pair`: the nearest one written among its own and
// those of the kLruLook - 1 tiles before it (`near` of them in its sequence), taken through the maps of the tiles between.
// These are applied one by one, from the state on, as the tiles themselves do: wherever the state comes from, the bits are
// the same.  BACK: the tiles that come before are those behind.  A wait that runs out sets the error word and goes on with
// zeros.
template <bool BACK>
__device__ __forceinline__ F2 look_back(const LruChain& c, const LruTile& t, unsigned cols, int pair, unsigned near) {
    const int64_t at = ((int64_t)t.number * cols + t.col) * kLruPairs + pair;
    const int64_t step = (BACK ? 1 : -1) * (int64_t)cols * kLruPairs;
    for (int poll = 0; poll < kLruPolls; ++poll) {
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
        F2 state = 0;
        int from = 0;
#pragma unroll
        for (int j = 0; j < kLruLook; ++j) {
            if (!found && linked && is_written(s[j])) found = true, state = s[j], from = j;
            linked = linked && is_written(m[j].x) && is_written(m[j].y);
        }
        if (__all_sync(0xffffffffu, found)) {
#pragma unroll
            for (int j = kLruLook - 2; j >= 0; --j)
                if (j < from) state = fma2(m[j].x, state, m[j].y);
            return state;
        }
        if ((poll & 4095) == 4095 && *reinterpret_cast<volatile unsigned*>(c.err)) break;
    }
    if ((threadIdx.x & 31) == 0) atomicCAS(c.err, 0u, kDeviceErrTimeout);
    return 0;
}

// What the guide tells the workers of a tile: three in turn, the next one's already known.
struct LruPlan {
    LruTile t;
    bool live;               // there is one
    alignas(8) float rates[kLruCols];
};
template <bool BACK, bool RATE>
__device__ __forceinline__ void lru_plan(const Lru& p, const LruChain& c, unsigned turn, LruPlan* plan) {
    const int lane = threadIdx.x & 31;
    const unsigned ticket = __shfl_sync(0xffffffffu, lane == 0 ? take_ticket(c, turn) : 0, 0);
    const bool live = ticket < p.tiles * p.cols;
    if (lane == 0) plan->live = live;
    if (!live) return;
    const LruTile t = lru_tile<BACK>(p, ticket);
    if (lane == 0) plan->t = t;
    const int ch = t.col * kLruCols + lane;
    if (RATE) plan->rates[lane] = ch < p.D ? rate_of(p.lam[ch], p.c) : 0.f;
}

// ---------------------------------------------------------------- inputs

// Where a row of a tile lies in shared memory.  Rows of 16-bit types, half a turn of the banks long, change places in every
// second run, so that the two runs of a warp read different banks.
template <typename IO> __device__ __forceinline__ int lru_place(int row) {
    return (sizeof(IO) == 2 ? row ^ (row / kLruRun & 1) : row) * kLruCols;
}
template <int BYTES> __device__ __forceinline__ void lru_copy(void* to, const void* from, int bytes) {
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
    if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(from), "r"(bytes) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(at), "l"(from), "r"(bytes) : "memory");
}
template <typename IO, int BYTES>
__device__ __forceinline__ void lru_fetch_units(const LruRows& v, const LruTile& t, int D, IO* to) {
    constexpr int per = BYTES / (int)sizeof(IO), pieces = kLruCols / per, step = kLruWorkers / pieces;
    const int piece = threadIdx.x % pieces, ch = t.col * kLruCols + piece * per;
    const int bytes = min(per, D - ch) * (int)sizeof(IO);
    if (bytes <= 0) return;
    const IO* from = (const IO*)v.p + (t.first + threadIdx.x / pieces) * v.ld + ch;
#pragma unroll
    for (int k = 0; k < kLruTile / step; ++k) {
        const int row = threadIdx.x / pieces + k * step;
        if (row < t.len) lru_copy<BYTES>(to + lru_place<IO>(row) + piece * per, from, bytes);
        from += step * v.ld;
    }
}
// A tile of a tensor on its way into shared memory, by the workers; rows past the tile's end stay what they were.
template <typename IO> __device__ __forceinline__ void lru_fetch(const LruRows& v, const LruTile& t, int D, IO* to) {
    if (v.unit == 16) {
        lru_fetch_units<IO, 16>(v, t, D, to);
    } else if (sizeof(IO) == 4 || v.unit == 4) {
        lru_fetch_units<IO, 4>(v, t, D, to);
    } else {
        constexpr int step = kLruWorkers / kLruPairs, most = kLruTile / step;
        const int piece = threadIdx.x % kLruPairs, ch = t.col * kLruCols + piece * 2, row0 = threadIdx.x / kLruPairs;
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
            *reinterpret_cast<RawN<IO, 2>*>(to + lru_place<IO>(row0 + k * step) + piece * 2) = e[k];
    }
}

// A token of the thread's run, two channels; past the tile's end anything.
template <typename IO> __device__ __forceinline__ F2 lru_read(const IO* from, int row, int pair) {
    return wide2(*reinterpret_cast<const RawN<IO, 2>*>(from + lru_place<IO>(row) + pair * 2));
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
inline Lru lru_of(const LruArgs& a, const LruTensors& t) {
    const int64_t e = a.io == GDR_F32 ? 4 : 2;
    Lru k{};
    k.q = Seqs{a.cu, a.total, a.T, (int)a.n};
    k.D = a.D;
    k.cols = (unsigned)((a.D + kLruCols - 1) / kLruCols);
    k.tiles = (unsigned)lru_tiles(a);
    k.x = lru_rows(t.x, e);
    k.r = lru_rows(t.r, e);
    k.i = lru_rows(t.i, e);
    k.lam = t.lam;
    k.h0 = t.h0;
    k.c = a.c;
    return k;
}

// The chain's words in the workspace, set to "not written"; with one tile a sequence there is none.
inline bool lru_one_tile_each(const LruArgs& a) { return (a.cu ? a.total : a.T) <= kLruTile; }
inline cudaError_t lru_chain(const LruArgs& a, void* workspace, LruChain* c, cudaStream_t s) {
    *c = LruChain{};
    if (lru_one_tile_each(a)) return cudaSuccess;
    const int64_t tiles = lru_tiles(a), cols = (a.D + kLruCols - 1) / kLruCols;
    c->ticket = (unsigned*)workspace;
    c->maps = (ulonglong2*)((char*)workspace + 256);
    c->states = (F2*)(c->maps + tiles * cols * kLruPairs);
    if (cudaError_t e = device_error_ptr(&c->err)) return e;
    return cudaMemsetAsync(workspace, 0xff, lru_chain_bytes(tiles, cols), s);
}

}  // namespace layer
}  // namespace gdr
