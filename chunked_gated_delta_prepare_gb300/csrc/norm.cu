// The root-mean-square norm of a row with the residual's addition, an 8-bit output with scales, and its gradient.
//
//   s = x + residual,  y = s w / sqrt(mean s^2 + eps)          (all in fp32, rounded once into r = s, y or y8)
//   y8 = e4m3(y / scale),  scale = max(amax / 448, 2^-126) over the row or over groups of its columns
//
// Bound: memory.  A row is read once and stays in registers (up to 4 vectors of 8 columns a thread) between the sum of
// squares and the output; w stays in registers over all the rows of a block, whose next row is in flight while it works
// on this one.  A row is held by 32 threads up to 1024
// columns (four rows a block, sums by shuffles alone), by a block above that.  With fewer rows than the GPU has room
// for blocks, a row is spread over more threads, one vector each, since then only the latency of one row counts.
//
// Gradient, with xh = s rstd and the sum taken over the row:
//   ds = rstd (w dy - xh mean(w dy xh)) + dr,   dw = sum over rows of dy xh
// One pass over dy and r: both sums of a row come from registers.  Each block adds its rows' dw in registers and
// leaves one row of partial sums, which column_sum adds in a fixed order: no atomics, the same bits in every run.
#include <cuda_fp8.h>

#include <algorithm>

#include "layer_common.cuh"
#include "layer_internal.h"

namespace gdr {
namespace layer {
namespace {

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
        for (int o = W / 2; o > 0; o >>= 1) {
            const float t = __shfl_xor_sync(0xffffffffu, u, o);
            u = MAX ? max_nan(u, t) : u + t;
        }
        v[i] = __shfl_sync(0xffffffffu, u, 0);
    }
}

__device__ __forceinline__ void store_e4m3(uint8_t* p, const float (&y)[8], float inv, int left, bool vec) {
    __nv_fp8x2_storage_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        q[i] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * i] * inv, y[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    if (vec && left >= 8) {
        *reinterpret_cast<uint2*>(p) =
            make_uint2((uint32_t)q[0] | (uint32_t)q[1] << 16, (uint32_t)q[2] | (uint32_t)q[3] << 16);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[i] = (uint8_t)(q[i >> 1] >> (8 * (i & 1)));
    }
}

// The backward's rows: dy, r and dr of the next RING - 1 rows of a block are on their way into shared memory, each
// thread's vectors in its own places, while the block works on one.  (With one row ahead in registers, as the forward
// has it, the kernel took twice the time; the forward's two tensors are faster that way, 20 against 28 us at 8192 x
// 2048.)  RING = 1: a row is loaded when it is its turn (few rows, rows not aligned, or rows too wide for the ring).
constexpr int kRingBytes = 56 * 1024;     // of a block, so that three or more fit an SM
template <typename IO, int NT, int VPT> constexpr int ring_of() {
    constexpr int row = NT * VPT * 3 * (int)sizeof(Raw8<IO>);
    return 4 * row <= kRingBytes ? 4 : 3 * row <= kRingBytes ? 3 : 2 * row <= kRingBytes ? 2 : 1;
}

template <typename IO, int NT, int VPT, int RING> struct Pipe {
    const IO* base[3];            // the tensors, or nullptr
    int64_t rows;
    int D, tid, tpr;
    bool vec;
    uint4* ring;                  // [RING][3][VPT][16-byte pieces of a vector][NT]

    __device__ __forceinline__ uint4* place(int slot, int t, int i, int part) const {
        constexpr int parts = sizeof(IO) / 2;
        return ring + ((((slot * 3 + t) * VPT + i) * parts + part) * NT + threadIdx.x);
    }
    // Starts row `row` towards its slot; a row that does not exist starts nothing.
    __device__ __forceinline__ void ahead(int64_t row, int slot) const {
        if (row < rows)
#pragma unroll
            for (int t = 0; t < 3; ++t)
                if (base[t])
#pragma unroll
                    for (int i = 0; i < VPT; ++i) {
                        const int c = (tid + i * tpr) * 8;
                        if (c < D)
#pragma unroll
                            for (int part = 0; part < (int)sizeof(IO) / 2; ++part)
                                copy_ahead(reinterpret_cast<RawN<IO, 16 / sizeof(IO)>*>(place(slot, t, i, part)),
                                           base[t] + row * D + c + part * (16 / (int)sizeof(IO)));
                    }
        copy_group();
    }
    // The thread's vectors of tensor t of the row; zeros past the row's end and for a row that does not exist.
    __device__ __forceinline__ void take(int64_t row, int slot, int t, Raw8<IO> (&v)[VPT]) const {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * tpr) * 8, left = row < rows ? D - c : 0;
            if (RING == 1) {
                v[i] = load8(base[t] + row * D + c, left, vec, c);
            } else if (left > 0) {
#pragma unroll
                for (int part = 0; part < (int)sizeof(IO) / 2; ++part)
                    reinterpret_cast<uint4*>(&v[i])[part] = *place(slot, t, i, part);
            } else {
                v[i] = load8((const IO*)nullptr, 0, false);
            }
        }
    }
};

// Blocks an SM that a kernel's registers leave room for: 1024 threads at one vector a thread, 768 at two (1024 spill and
// take 179 us instead of 160 for 32768 x 4096 to e4m3, 512 take 188), 512 at four.
template <int TPR, int VPT> constexpr int blocks_per_sm() {
    constexpr int threads = VPT > 2 ? 512 : VPT > 1 ? 768 : 1024, nt = TPR < 128 ? 128 : TPR;
    return threads > nt ? threads / nt : 1;
}

template <typename IO, int TPR, int VPT>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR, blocks_per_sm<TPR, VPT>())
norm_forward_kernel(NormArgs a, RowTensor x, RowTensor res, const IO* __restrict__ w, IO* __restrict__ y,
                    IO* __restrict__ r, uint8_t* __restrict__ y8, float* __restrict__ scales, bool vec_w, bool vec_y,
                    bool vec_r, bool vec_8) {
    constexpr int RPB = TPR < 128 ? 128 / TPR : 1;
    __shared__ float red[2 * 32], redm[2 * 32];
    const int tid = threadIdx.x % TPR, slot = threadIdx.x / TPR;
    const int D = a.D;
    Raw8<IO> wr[VPT], xr[VPT], sr[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (tid + i * TPR) * 8;
        wr[i] = load8(w + c, D - c, vec_w);
    }
    const bool two = res.p != nullptr;
    const auto fetch = [&](int64_t row) {     // a block's last rows may not exist: zeros
        const IO* xp = reinterpret_cast<const IO*>(x.p) + row * x.ld;
        const IO* sp = reinterpret_cast<const IO*>(res.p) + row * res.ld;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * TPR) * 8, left = row < a.rows ? D - c : 0;
            xr[i] = load8(xp + c, left, x.vec, c);
            if (two) sr[i] = load8(sp + c, left, res.vec, c);
        }
    };
    fetch((int64_t)blockIdx.x * RPB + slot);
    int turn = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < a.rows; row0 += (int64_t)gridDim.x * RPB, ++turn) {
        const int64_t row = row0 + slot;
        const bool live = row < a.rows;       // threads of a row that does not exist stay for the shuffles
        float v[VPT][8], sum[1] = {0.f};
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            widen(xr[i], v[i]);
            if (two) {
                float t[8];
                widen(sr[i], t);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += t[j];
            }
        }
        fetch(row + (int64_t)gridDim.x * RPB);          // in flight while this row is worked on
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * TPR) * 8;
            if (r) store_n(r + row * D + c, v[i], live ? D - c : 0, vec_r);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[0] = fmaf(v[i][j], v[i][j], sum[0]);
        }
        row_reduce<TPR, 1, false>(sum, red, turn);
        const float rstd = rsqrtf(sum[0] / (float)D + a.eps);
        float top[1] = {0.f};
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * TPR) * 8;
            float wf[8], m = 0.f;
            widen(wr[i], wf);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] = v[i][j] * rstd * wf[j];
                if (y8) m = max_nan(m, fabsf(v[i][j]));  // zero past the row's end, or NaN in a row of nothing else
            }
            if (y) store_n(y + row * D + c, v[i], live ? D - c : 0, vec_y);
            if (y8 && a.group) {             // a group's columns lie in group / 8 neighbouring threads
                for (int o = a.group / 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                const float scale = max_nan(m * (1.f / 448.f), 1.17549435e-38f);
                if (live && c < D) {
                    store_e4m3(y8 + row * D + c, v[i], 1.f / scale, D - c, vec_8);
                    if ((c & (a.group - 1)) == 0)
                        scales[row * ((D + a.group - 1) / a.group) + c / a.group] = scale;
                }
            }
            top[0] = max_nan(top[0], m);
        }
        if (y8 && !a.group) {
            row_reduce<TPR, 1, true>(top, redm, turn);
            const float scale = max_nan(top[0] * (1.f / 448.f), 1.17549435e-38f), inv = 1.f / scale;
            if (live) {
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const int c = (tid + i * TPR) * 8;
                    store_e4m3(y8 + row * D + c, v[i], inv, D - c, vec_8);
                }
                if (tid == 0) scales[row] = scale;
            }
        }
    }
}

template <typename IO, int TPR, int VPT, int RING>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR, blocks_per_sm<TPR, VPT>() > 1 ? blocks_per_sm<TPR, VPT>() / 2 : 1)
norm_backward_kernel(NormArgs a, const IO* __restrict__ dy, const IO* __restrict__ r, const IO* __restrict__ w,
                     const IO* __restrict__ dr, IO* __restrict__ dx, float* __restrict__ partial, bool vec) {
    constexpr int RPB = TPR < 128 ? 128 / TPR : 1, NT = TPR * RPB;
    extern __shared__ uint4 smem[];
    __shared__ float red[2 * 2 * 32];
    const int tid = threadIdx.x % TPR, slot = threadIdx.x / TPR;
    const int D = a.D;
    Raw8<IO> wr[VPT];
    float dw[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (tid + i * TPR) * 8;
        wr[i] = load8(w + c, D - c, vec);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
    }
    const int64_t step = (int64_t)gridDim.x * RPB, first = (int64_t)blockIdx.x * RPB + slot;
    const Pipe<IO, NT, VPT, RING> in{{dy, r, dr}, a.rows, D, tid, TPR, vec, smem};
#pragma unroll
    for (int k = 0; k < RING - 1; ++k) in.ahead(first + k * step, k);
    int turn = 0, at = 0;
    for (int64_t row = first; row - slot < a.rows; row += step, ++turn, at = at + 1 == RING ? 0 : at + 1) {
        const bool live = row < a.rows;
        Raw8<IO> yr[VPT], rr[VPT];
        if (RING > 1) {
            in.ahead(row + (RING - 1) * step, at == 0 ? RING - 1 : at - 1);
            copy_wait<RING - 1>();
        }
        in.take(row, at, 0, yr);
        in.take(row, at, 1, rr);
        float sum[2] = {0.f, 0.f};            // of s^2 and of w dy s
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float s[8], g[8], wf[8];
            widen(rr[i], s), widen(yr[i], g), widen(wr[i], wf);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sum[0] = fmaf(s[j], s[j], sum[0]);
                sum[1] = fmaf(wf[j] * g[j], s[j], sum[1]);
            }
        }
        row_reduce<TPR, 2, false>(sum, red, turn);
        const float rstd = rsqrtf(sum[0] / (float)D + a.eps);
        const float back = sum[1] / (float)D * rstd * rstd;
        Raw8<IO> er[VPT];
        if (dr) in.take(row, at, 2, er);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * TPR) * 8;
            float s[8], g[8], wf[8], o[8];
            widen(rr[i], s), widen(yr[i], g), widen(wr[i], wf);
            if (dr) widen(er[i], o);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                o[j] = fmaf(rstd, fmaf(-s[j], back, wf[j] * g[j]), dr ? o[j] : 0.f);
                if (live) dw[i][j] = fmaf(g[j], s[j] * rstd, dw[i][j]);
            }
            if (live) store_n(dx + row * D + c, o, D - c, vec);
        }
    }
    float* mine = partial + ((int64_t)blockIdx.x * RPB + slot) * D;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (tid + i * TPR) * 8;
        store_n(mine + c, dw[i], D - c, (D & 3) == 0);
    }
}

// 32 columns a block, 32 rows in flight; the 32 partial sums of a column are added in shared memory in order.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* __restrict__ in, int64_t rows, int64_t ld,
                                                          int64_t cols, float* __restrict__ out, int64_t cols2,
                                                          float* __restrict__ out2) {
    __shared__ float part[32][33];
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (c < cols + cols2) {
#pragma unroll 8
        for (int64_t i = threadIdx.y; i < rows; i += 32) s += in[i * ld + c];
    }
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    float t = part[threadIdx.x][threadIdx.y];      // warp y adds column y
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    const int64_t cc = (int64_t)blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && cc < cols) out[cc] = t;
    else if (threadIdx.x == 0 && cc < cols + cols2) out2[cc - cols] = t;
}

// Threads of a row and vectors a thread.  Many rows: few threads with up to 4 vectors each.  Few rows (less than two
// blocks an SM): one vector each, as far as a block reaches.
struct Shape {
    int tpr, vpt;
};
Shape shape_of(const NormArgs& a) {
    const int v = (a.D + 7) / 8;
    if (v <= 32) return {32, 1};
    const bool few = a.rows < 2 * kSms;
    if (!few && v <= 64) return {32, 2};
    if (!few && v <= 128) return {32, 4};
    if (few)
        for (int tpr = 128; tpr <= 1024; tpr *= 2)
            if (v <= tpr) return {tpr, 1};
    if (few && v <= 2048) return {1024, 2};
    if (v <= 256) return {128, 2};
    if (v <= 512) return {256, 2};
    return {v <= 1024 ? 256 : v <= 2048 ? 512 : 1024, 4};
}

template <typename IO, int TPR, int VPT>
cudaError_t launch_forward(const NormArgs& a, RowTensor x, RowTensor res, const void* w, void* y, void* r, void* y8,
                           float* scales, cudaStream_t s) {
    constexpr int RPB = TPR < 128 ? 128 / TPR : 1, NT = TPR < 128 ? 128 : TPR;
    const int64_t blocks = (a.rows + RPB - 1) / RPB;
    const int grid = (int)std::min<int64_t>(blocks, (int64_t)kSms * blocks_per_sm<TPR, VPT>());
    const auto al = [&](const void* p, int unit) {
        return (reinterpret_cast<uintptr_t>(p) % 16) == 0 && ((int64_t)a.D * unit) % 16 == 0;
    };
    norm_forward_kernel<IO, TPR, VPT><<<grid, NT, 0, s>>>(
        a, x, res, (const IO*)w, (IO*)y, (IO*)r, (uint8_t*)y8, scales, reinterpret_cast<uintptr_t>(w) % 16 == 0,
        al(y, sizeof(IO)), al(r, sizeof(IO)), reinterpret_cast<uintptr_t>(y8) % 8 == 0 && a.D % 8 == 0);
    return cudaGetLastError();
}

// The gradient's: one vector a thread as far as 512 threads reach, since its sums of dw and two rows' inputs fill the
// registers at two (30 us instead of 24 at 8192 x 2048).
Shape backward_shape(const NormArgs& a) {
    const int v = (a.D + 7) / 8;
    if (v > 32)
        for (int tpr = 128; tpr <= 512; tpr *= 2)
            if (v <= tpr) return {tpr, 1};
    return shape_of(a);
}

// One wave of the gradient's blocks: half the forward's threads an SM, for the sums of dw in registers.
int64_t backward_grid(const NormArgs& a, Shape h) {
    const int rpb = h.tpr < 128 ? 128 / h.tpr : 1, nt = h.tpr < 128 ? 128 : h.tpr;
    return std::min<int64_t>((a.rows + rpb - 1) / rpb, (int64_t)kSms * std::max(1, (h.vpt > 2 ? 256 : 512) / nt));
}

template <typename IO, int TPR, int VPT>
cudaError_t launch_backward(const NormArgs& a, const void* dy, const void* r, const void* w, const void* dr, void* dx,
                            float* partial, cudaStream_t s) {
    constexpr int RPB = TPR < 128 ? 128 / TPR : 1, NT = TPR < 128 ? 128 : TPR, RING = ring_of<IO, NT, VPT>();
    bool vec = ((int64_t)a.D * sizeof(IO)) % 16 == 0;
    for (const void* p : {dy, r, w, dr, (const void*)dx}) vec = vec && reinterpret_cast<uintptr_t>(p) % 16 == 0;
    const int64_t grid = backward_grid(a, {TPR, VPT});
    const auto go = [&](auto ring) {
        constexpr int R = decltype(ring)::value, bytes = R > 1 ? R * NT * VPT * 3 * (int)sizeof(Raw8<IO>) : 0;
        const auto kernel = norm_backward_kernel<IO, TPR, VPT, R>;
        if (bytes > 40 * 1024)
            if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) return e;
        kernel<<<(unsigned)grid, NT, bytes, s>>>(a, (const IO*)dy, (const IO*)r, (const IO*)w, (const IO*)dr, (IO*)dx,
                                                 partial, vec);
        return cudaGetLastError();
    };
    if (RING > 1 && a.D % 8 == 0 && vec && grid * RPB < a.rows) return go(std::integral_constant<int, RING>());
    return go(std::integral_constant<int, 1>());
}

// Calls f with the shape's constants.
template <bool BACKWARD, typename F> cudaError_t with_shape(Shape h, F f) {
#define GDR_SHAPE(T, V) \
    if (h.tpr == T && h.vpt == V) return f(std::integral_constant<int, T>(), std::integral_constant<int, V>());
    GDR_SHAPE(32, 1)
    GDR_SHAPE(128, 1) GDR_SHAPE(256, 1) GDR_SHAPE(512, 1) GDR_SHAPE(1024, 1) GDR_SHAPE(1024, 2)
    GDR_SHAPE(256, 4) GDR_SHAPE(512, 4) GDR_SHAPE(1024, 4)
    if constexpr (!BACKWARD) {
        GDR_SHAPE(32, 2) GDR_SHAPE(32, 4)
        GDR_SHAPE(128, 2) GDR_SHAPE(256, 2)
    }
#undef GDR_SHAPE
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t norm_forward(const NormArgs& a, RowTensor x, RowTensor res, const void* w, void* y, void* r, void* y8,
                         float* scales, cudaStream_t s) {
    return with_shape<false>(shape_of(a), [&](auto tpr, auto vpt) {
        constexpr int T = decltype(tpr)::value, V = decltype(vpt)::value;
        if (a.io == GDR_F32) return launch_forward<float, T, V>(a, x, res, w, y, r, y8, scales, s);
        if (a.io == GDR_BF16) return launch_forward<__nv_bfloat16, T, V>(a, x, res, w, y, r, y8, scales, s);
        return launch_forward<__half, T, V>(a, x, res, w, y, r, y8, scales, s);
    });
}

int64_t norm_partial_rows(const NormArgs& a) {
    const Shape h = backward_shape(a);
    return backward_grid(a, h) * (h.tpr < 128 ? 128 / h.tpr : 1);
}

cudaError_t norm_backward(const NormArgs& a, const void* dy, const void* r, const void* w, const void* dr, void* dx,
                          float* dw, float* partial, cudaStream_t s) {
    const cudaError_t e = with_shape<true>(backward_shape(a), [&](auto tpr, auto vpt) {
        constexpr int T = decltype(tpr)::value, V = decltype(vpt)::value;
        if (a.io == GDR_F32) return launch_backward<float, T, V>(a, dy, r, w, dr, dx, partial, s);
        if (a.io == GDR_BF16) return launch_backward<__nv_bfloat16, T, V>(a, dy, r, w, dr, dx, partial, s);
        return launch_backward<__half, T, V>(a, dy, r, w, dr, dx, partial, s);
    });
    if (e != cudaSuccess) return e;
    return column_sum(partial, norm_partial_rows(a), a.D, a.D, dw, 0, nullptr, s);
}

cudaError_t column_sum(const float* in, int64_t rows, int64_t ld, int64_t cols, float* out, int64_t cols2, float* out2,
                       cudaStream_t s) {
    if (cols + cols2 <= 0) return cudaSuccess;
    column_sum_kernel<<<(unsigned)((cols + cols2 + 31) / 32), dim3(32, 32), 0, s>>>(in, rows, ld, cols, out, cols2,
                                                                                    out2);
    return cudaGetLastError();
}

}  // namespace layer
}  // namespace gdr
