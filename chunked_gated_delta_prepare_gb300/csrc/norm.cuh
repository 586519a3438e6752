// What the norm's forward and gradient share: sums over a row's threads, rows that do not start on 16-byte boundaries, and
// the blocks of a wave.
#pragma once

#include <algorithm>

#include "layer_common.cuh"
#include "layer_internal.h"

namespace gdr {
namespace layer {

// Sums of v[0..NV) over the TPR threads of a row.  red: [2][NV][32] floats, the halves used in turn so that one
// barrier a row is enough.
template <int TPR, int NV, bool MAX>
__device__ __forceinline__ void row_reduce(float (&v)[NV], float* red, int turn) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const float u = __shfl_xor_sync(0xffffffffu, v[i], o);
            v[i] = MAX ? max_nan(v[i], u) : v[i] + u;
        }
    if (TPR == 32) return;
    constexpr int W = TPR / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* mine = red + (turn & 1) * NV * 32;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < NV; ++i) mine[i * 32 + warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float u = lane < W ? mine[i * 32 + lane] : 0.f;   // both the squares' sum and a largest absolute value are >= 0
#pragma unroll
        for (int o = W > 16 ? 16 : W > 8 ? 8 : W > 4 ? 4 : 2; o > 0; o >>= 1) {
            const float t = __shfl_xor_sync(0xffffffffu, u, o);
            u = MAX ? max_nan(u, t) : u + t;
        }
        v[i] = __shfl_sync(0xffffffffu, u, 0);
    }
}

// Where a contiguous row of D elements starts between two 16-byte boundaries, the tensor starting on one, in elements.
template <typename IO> __device__ __forceinline__ int first_shift(int64_t row, int D) {
    constexpr int per = 16 / (int)sizeof(IO);
    return (int)(row % per * (D % per) % per);
}

// Rows that do not start on 16-byte boundaries.  Where all tensors of a call share the place `shift` of a row's first
// element between two boundaries (contiguous rows of D elements that are no multiple of 16 bytes), a thread's vectors are
// cut at the boundaries instead of at column 0: vector i of a row covers the columns from 8 i - shift on, and only a row's
// first and last vector are not whole.  The shift returns after `period` rows, so with a multiple of that many
// rows from one turn to the next it is a block's own, and w and the sums of dw stay in registers as for aligned rows.
// (16384 rows of 4089 columns to e4m3: fp32 434 us with vectors from column 0 on, 158 cut, 137 with 4096 columns; bf16
// 214, 85 and 75.)

// Whether the vector that starts at column c < D of a row ends past the tensor of `rows` rows.  In rows narrower than a
// vector that is so in several of the tensor's last rows (up to 8: a vector has no more columns), not in the very last alone.
__host__ __device__ __forceinline__ bool ends_past(int64_t row, int64_t rows, int c, int D) {
    return rows - row <= 8 && c + 8 > (int)(rows - row) * D;
}
// Elements [at, at + 8) of a tensor of `total`, or any vector where they are not all in it.  A row's first and last vector
// bring the neighbour rows' elements along; mask_cut takes them out when they are used, and a vector that ends past the
// tensor is loaded then.  Done on arrival, both would read or write the registers that the load fills, and keep the warp,
// and at its barrier the block, waiting for memory in every row.
template <typename IO> __device__ __forceinline__ Raw8<IO> load_around(const IO* p, int64_t at, int64_t total) {
    return load8(p + (at + 8 <= total ? at : 0), 8, true);
}
// Elements [c, c + 8) of a row, zeros outside it.
template <typename IO> __device__ __forceinline__ Raw8<IO> load_cut(const IO* row, int c, int D, bool vec) {
    if (vec && c >= 0 && c + 8 <= D) return load8(row + c, 8, true);
    Raw8<IO> r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.e[i] = c + i >= 0 && c + i < D ? row[c + i] : from_f<IO>(0.f);
    return r;
}
// Elements [lo, hi) of an aligned vector at p, either lo = 0 or hi = 8.
template <typename IO> __device__ __forceinline__ void store_piece(IO* p, const Raw8<IO>& r, int lo, int hi) {
    using Four = RawN<IO, 4>;
    using Two = RawN<IO, 2>;
#pragma unroll
    for (int i = 0; i < 8; i += 4)
        if (i >= lo && i + 4 <= hi) *reinterpret_cast<Four*>(p + i) = *reinterpret_cast<const Four*>(r.e + i);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {           // a half of a quarter that is not whole
        const bool four = (i & 4) >= lo && (i & 4) + 4 <= hi;
        if (!four && i >= lo && i + 2 <= hi) *reinterpret_cast<Two*>(p + i) = *reinterpret_cast<const Two*>(r.e + i);
        if (i + 1 == lo) p[i + 1] = r.e[i + 1];
        if (i + 1 == hi) p[i] = r.e[i];
    }
}
template <typename IO> __device__ __forceinline__ void mask_cut(Raw8<IO>& r, int c, int D) {
    if (c < 0 || c + 8 > D)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < 0 || c + i >= D) r.e[i] = from_f<IO>(0.f);
}
// vec: column c lies on a 16-byte boundary, so what a row has of its first or last vector goes in pieces of 4, 2 and 1.
template <typename IO> __device__ __forceinline__ void store_cut(IO* row, const float (&x)[8], int c, int D, bool vec) {
    Raw8<IO> r;
#pragma unroll
    for (int i = 0; i < 8; i += 2) from_f2(r.e + i, x[i], x[i + 1]);
    if (c >= 0 && c + 8 <= D) {
        store_raw(row + c, r, 8, vec);
    } else if (vec && (c >= 0 || c + 8 <= D)) {
        store_piece(row + c, r, c < 0 ? -c : 0, c < 0 ? 8 : D - c);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i >= 0 && c + i < D) row[c + i] = r.e[i];
    }
}

// Blocks an SM that a kernel's registers leave room for: 1024 threads at one vector a thread, 800 at two (with 256 a block
// that is 768: 164 us for 32768 x 4096 to e4m3; 1024 spill and take 179, 512 take 188), 512 at four.
template <int TPR, int VPT> constexpr int blocks_per_sm() {
    constexpr int threads = VPT > 2 ? 512 : VPT > 1 ? 800 : 1024, nt = TPR < 128 ? 128 : TPR;
    return threads > nt ? threads / nt : 1;
}

// a.D + 7: cut at the boundaries a row may touch one vector more (in the longest rows one more than a block holds; they
// are not cut).
inline int vectors_of(const NormArgs& a) {
    return (a.D + (a.D * (a.io == GDR_F32 ? 4 : 2) % 16 ? 14 : 7)) / 8;
}

// Threads of a row and vectors a thread.
struct Shape {
    int tpr, vpt;
};

}  // namespace layer
}  // namespace gdr
