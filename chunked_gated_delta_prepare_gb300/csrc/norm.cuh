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
// first and last vector go element by element.  The shift returns after `period` rows, so with a multiple of that many
// rows from one turn to the next it is a block's own, and w and the sums of dw stay in registers as for aligned rows.
// (16384 rows of 4089 instead of 4096 columns: fp32 434 us before, 141 now, 137 aligned; bf16 214, 167 and 75.)
// Elements [c, c + 8) of a row, which may begin before its first or end past its last element: those read as zero, or, in
// a vector that lies in the tensor all the same (`more`: rows follow this one), as what is there, for mask_cut to take
// out when it is used.  (Taken out on arrival, they would keep their warp, and at its barrier the block, waiting for
// memory in every row.)
template <typename IO> __device__ __forceinline__ Raw8<IO> load_cut(const IO* row, int c, int D, bool vec, bool more) {
    if (vec && c < D && (more || c + 8 <= D)) return load8(row + c, 8, true);   // c < 0: the end of the row before
    Raw8<IO> r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.e[i] = c + i >= 0 && c + i < D ? row[c + i] : from_f<IO>(0.f);
    return r;
}
template <typename IO> __device__ __forceinline__ void mask_cut(Raw8<IO>& r, int c, int D) {
    if (c < 0 || c + 8 > D)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < 0 || c + i >= D) r.e[i] = from_f<IO>(0.f);
}
template <typename IO> __device__ __forceinline__ void store_cut(IO* row, const float (&x)[8], int c, int D, bool vec) {
    if (c >= 0) {
        store_n(row + c, x, D - c, vec);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i >= 0 && c + i < D) row[c + i] = from_f<IO>(x[i]);
    }
}

// Blocks an SM that a kernel's registers leave room for: 1024 threads at one vector a thread, 768 at two (1024 spill and
// take 179 us instead of 160 for 32768 x 4096 to e4m3, 512 take 188), 512 at four.
template <int TPR, int VPT> constexpr int blocks_per_sm() {
    constexpr int threads = VPT > 2 ? 512 : VPT > 1 ? 768 : 1024, nt = TPR < 128 ? 128 : TPR;
    return threads > nt ? threads / nt : 1;
}

// a.D + 7: cut at the boundaries (see load_cut) a row may touch one vector more.
inline int vectors_of(const NormArgs& a) {
    return (a.D + (a.D * (a.io == GDR_F32 ? 4 : 2) % 16 ? 14 : 7)) / 8;
}

// Threads of a row and vectors a thread.
struct Shape {
    int tpr, vpt;
};

}  // namespace layer
}  // namespace gdr
