// Device helpers shared by the layer operators (norm, convolution, selective scan, single-token delta step).
//
// They work on vectors of 8 (or 4) neighbouring channels of one token.  A row may start at any element: where its
// address is not a multiple of 16 bytes, the scan and the norm's fp32 gradient take a vector from the aligned blocks around
// it (4 times fewer trips through the L1 cache than element by element), the convolution by words; the norm cuts contiguous
// rows at the boundaries and takes slices element by element (see norm.cu).  Vectors go out in aligned words; at a row's
// ends the elements move one by one.
// Whether a tensor's rows are all aligned is decided on the host (RowTensor::vec).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gdr {
namespace layer {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <typename IO> __device__ __forceinline__ IO from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }

// N neighbouring elements as they lie in memory.
template <typename IO, int N> struct alignas(sizeof(IO) * N < 16 ? sizeof(IO) * N : 16) RawN {
    IO e[N];
};
template <typename IO> using Raw8 = RawN<IO, 8>;

// A vector that starts `off` bytes into aligned blocks, from the blocks' words (the last one is only ever shifted out).
template <int N, typename IO, int WORDS> __device__ __forceinline__ RawN<IO, N> shift_words(uint32_t (&w)[WORDS], int off) {
    if (WORDS > N * (int)sizeof(IO) / 4 + 3 && (off & 8))
#pragma unroll
        for (int i = 0; i < WORDS - 2; ++i) w[i] = w[i + 2];
    if (off & 4)
#pragma unroll
        for (int i = 0; i < WORDS - 1; ++i) w[i] = w[i + 1];
    RawN<IO, N> r;
#pragma unroll
    for (int i = 0; i < N * (int)sizeof(IO) / 4; ++i)
        reinterpret_cast<uint32_t*>(&r)[i] =
            sizeof(IO) == 4 ? w[i] : __funnelshift_r(w[i], w[i + 1], (off & 2) * 8);
    return r;
}

// A vector that starts at any element: the aligned blocks around it, shifted together.  Every block read must lie in the
// row, so a vector of it must come before and another after.
template <int N, typename IO> __device__ __forceinline__ RawN<IO, N> load_shifted(const IO* p) {
    constexpr int bytes = N * (int)sizeof(IO), block = bytes < 16 ? 8 : 16, words = (bytes + block) / 4;
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    const int off = (int)(at % block);
    uint32_t w[words + 1];
    w[words] = 0;
    if constexpr (block == 8) {
        const uint2* s = reinterpret_cast<const uint2*>(at - off);
#pragma unroll
        for (int i = 0; i < words / 2; ++i) *reinterpret_cast<uint2*>(w + 2 * i) = __ldg(s + i);
    } else {
        const uint4* s = reinterpret_cast<const uint4*>(at - off);
#pragma unroll
        for (int i = 0; i < words / 4; ++i) *reinterpret_cast<uint4*>(w + 4 * i) = __ldg(s + i);
    }
    return shift_words<N, IO>(w, off);
}

// Elements [0, N) of p; only the first `left` exist (left <= 0: none), the rest read as zero.  vec: the row starts on a
// 16-byte boundary, and so does p, or on one of its own size.  before: elements of the row in front of p.
template <int N, typename IO>
__device__ __forceinline__ RawN<IO, N> load_n(const IO* p, int64_t left, bool vec, int64_t before = 0) {
    RawN<IO, N> r;
    if (vec && left >= N) {
        if constexpr (sizeof(r) == 8) {
            *reinterpret_cast<uint2*>(&r) = __ldg(reinterpret_cast<const uint2*>(p));
        } else {
#pragma unroll
            for (int i = 0; i < (int)sizeof(r) / 16; ++i)
                reinterpret_cast<uint4*>(&r)[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
        }
    } else if (before >= N && left >= 2 * N) {
        r = load_shifted<N>(p);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) r.e[i] = i < left ? p[i] : from_f<IO>(0.f);
    }
    return r;
}

// The same for memory that the kernel also writes (not by way of the read-only cache).
template <int N, typename IO> __device__ __forceinline__ RawN<IO, N> load_own(const IO* p, int64_t left, bool vec) {
    RawN<IO, N> r;
    if (vec && left >= N) {
        if constexpr (sizeof(r) == 8) {
            *reinterpret_cast<uint2*>(&r) = *reinterpret_cast<const uint2*>(p);
        } else {
#pragma unroll
            for (int i = 0; i < (int)sizeof(r) / 16; ++i)
                reinterpret_cast<uint4*>(&r)[i] = reinterpret_cast<const uint4*>(p)[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) r.e[i] = i < left ? p[i] : from_f<IO>(0.f);
    }
    return r;
}
template <typename IO>
__device__ __forceinline__ Raw8<IO> load8(const IO* p, int64_t left, bool vec, int64_t before = 0) {
    return load_n<8>(p, left, vec, before);
}

// Two neighbours at a time: half the instructions of one by one.
__device__ __forceinline__ float2 to_f2(const float* p) { return make_float2(p[0], p[1]); }
__device__ __forceinline__ float2 to_f2(const __nv_bfloat16* p) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ float2 to_f2(const __half* p) { return __half22float2(*reinterpret_cast<const __half2*>(p)); }
__device__ __forceinline__ void from_f2(float* p, float a, float b) { p[0] = a, p[1] = b; }
__device__ __forceinline__ void from_f2(__nv_bfloat16* p, float a, float b) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
}
__device__ __forceinline__ void from_f2(__half* p, float a, float b) {
    *reinterpret_cast<__half2*>(p) = __floats2half2_rn(a, b);
}

template <typename IO, int N> __device__ __forceinline__ void widen(const RawN<IO, N>& r, float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 f = to_f2(r.e + i);
        x[i] = f.x, x[i + 1] = f.y;
    }
}

// An aligned vector on its way into the thread's own place in shared memory: no register holds it meanwhile.
template <typename IO, int N> __device__ __forceinline__ void copy_ahead(RawN<IO, N>* to, const IO* from) {
    static_assert(sizeof(RawN<IO, N>) == 8 || sizeof(RawN<IO, N>) == 16, "one copy");
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from),
                 "n"((int)sizeof(RawN<IO, N>))
                 : "memory");
}
// A word, of which `bytes` are read and the rest becomes zero.
__device__ __forceinline__ void copy_word(void* to, const void* from, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void copy_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT> __device__ __forceinline__ void copy_wait() {   // until at most LEFT groups are on their way
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

template <typename IO, int N>
__device__ __forceinline__ void store_raw(IO* p, const RawN<IO, N>& r, int64_t left, bool vec) {
    if (vec && left >= N) {
        if constexpr (sizeof(r) == 8) {
            *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(&r);
        } else {
#pragma unroll
            for (int i = 0; i < (int)sizeof(r) / 16; ++i)
                reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(&r)[i];
        }
    } else if (sizeof(IO) == 2 && left >= N) {          // whole words where they are aligned
        constexpr int words = N / 2;
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
        if ((reinterpret_cast<uintptr_t>(p) & 2) == 0) {
#pragma unroll
            for (int i = 0; i < words; ++i) reinterpret_cast<uint32_t*>(p)[i] = w[i];
        } else {
            p[0] = r.e[0];
#pragma unroll
            for (int i = 0; i < words - 1; ++i)
                reinterpret_cast<uint32_t*>(p + 1)[i] = __funnelshift_r(w[i], w[i + 1], 16);
            p[N - 1] = r.e[N - 1];
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < left) p[i] = r.e[i];
    }
}

template <typename IO, int N>
__device__ __forceinline__ void store_n(IO* p, const float (&x)[N], int64_t left, bool vec) {
    RawN<IO, N> r;
#pragma unroll
    for (int i = 0; i < N; i += 2) from_f2(r.e + i, x[i], x[i + 1]);
    store_raw(p, r, left, vec);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / (1 + e^-x): 0 and 1 at the ends of the range, NaN for NaN.
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + ex2(-x * kLog2e)); }

// Packed fp32: two independent operations an instruction, each rounded as alone.
using F2 = unsigned long long;   // the lower channel in the low half

__device__ __forceinline__ F2 pack2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpack2(F2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

template <typename IO, int N> __device__ __forceinline__ void pairs(const RawN<IO, N>& r, F2 (&v)[N / 2]) {
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
        const float2 f = to_f2(r.e + 2 * k);
        v[k] = pack2(f.x, f.y);
    }
}

__device__ __forceinline__ F2 both(float x) { return pack2(x, x); }
__device__ __forceinline__ F2 ex2_2(F2 v) {
    const float2 f = unpack2(v);
    return pack2(ex2(f.x), ex2(f.y));
}
__device__ __forceinline__ F2 rcp_2(F2 v) {
    const float2 f = unpack2(v);
    return pack2(rcp(f.x), rcp(f.y));
}
__device__ __forceinline__ F2 sigmoid2(F2 x) { return rcp_2(add2(both(1.f), ex2_2(mul2(x, both(-kLog2e))))); }

// silu of two, and its derivative
__device__ __forceinline__ F2 silu2(F2 p) { return mul2(p, sigmoid2(p)); }
__device__ __forceinline__ F2 silu_slope2(F2 p) {
    const F2 s = sigmoid2(p);
    return mul2(s, fma2(p, add2(both(1.f), mul2(s, both(-1.f))), both(1.f)));
}

__device__ __forceinline__ float max_nan(float a, float b) {   // NaN where either is
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// The packed sequences of a token axis, or a batch of equal ones (cu == nullptr: n rows of T tokens).
struct Seqs {
    const int* cu;    // device int32 [n + 1], or nullptr
    int64_t total;    // tokens on the axis
    int64_t T;        // tokens of each sequence of a batch
    int n;
};

// Sequence s as [start, start + len); whatever cu holds, the range lies in [0, total].
__device__ __forceinline__ void seq_range(const Seqs& q, int s, int64_t* start, int64_t* len) {
    if (!q.cu) {
        *start = (int64_t)s * q.T;
        *len = q.T;
        return;
    }
    int64_t a = q.cu[s], b = q.cu[s + 1];
    a = a < 0 ? 0 : (a > q.total ? q.total : a);
    b = b < a ? a : (b > q.total ? q.total : b);
    *start = a;
    *len = b - a;
}

// Tiles of `tile` tokens, numbered over all sequences.  Sequence s of a packed axis owns the numbers from
// cu[s] / tile + s up to cu[s + 1] / tile + s + 1 (its tiles and at most one more, which is empty), so the number of
// blocks, total / tile + n, needs no look at the lengths on the host.  A batch has ceil(T / tile) a sequence.
struct TileAt {
    int seq;          // -1: no such tile
    int64_t tile;     // within the sequence
    int64_t start, len;
};

__host__ __device__ __forceinline__ int64_t tile_count(const Seqs& q, int tile) {
    return q.cu ? q.total / tile + q.n : q.n * ((q.T + tile - 1) / tile);
}

__device__ __forceinline__ int64_t first_tile(const Seqs& q, int s, int tile) {
    if (!q.cu) return s * ((q.T + tile - 1) / tile);
    int64_t a = q.cu[s];
    a = a < 0 ? 0 : (a > q.total ? q.total : a);
    return a / tile + s;
}

__device__ __forceinline__ TileAt find_tile(const Seqs& q, int64_t number, int tile) {
    TileAt t;
    if (!q.cu) {
        const int64_t per = (q.T + tile - 1) / tile;
        t.seq = (int)(number / per);
        t.tile = number - t.seq * per;
        t.start = t.seq * q.T;
        t.len = q.T;
        return t;
    }
    int lo = 0, hi = q.n - 1;             // the last sequence whose first number is at most this one
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first_tile(q, mid, tile) <= number) lo = mid;
        else hi = mid - 1;
    }
    t.seq = lo;
    t.tile = number - first_tile(q, lo, tile);
    seq_range(q, lo, &t.start, &t.len);
    if (t.tile < 0 || (t.tile > 0 && t.tile * tile >= t.len)) t.seq = -1;
    return t;
}

}  // namespace layer
}  // namespace gdr
