// The root-mean-square norm of a row with the residual's addition, an 8-bit output with scales, and its gradient.
//
//   s = x + residual,  y = s w / sqrt(mean s^2 + eps)          (all in fp32, rounded once into r = s, y or y8)
//   y8 = e4m3(y / scale),  scale = max(amax / 448, 2^-126) over the row or over groups of its columns
//
// Bound: memory.  A row is read once and stays in registers (up to 4 vectors of 8 columns a thread) between the sum of
// squares and the output; w stays in registers over all the rows of a block, whose next row is in flight while it works
// on this one.  A row is held by 32 threads up to 1024 columns (four rows a block, sums by shuffles alone), by a block
// above that.  With fewer rows than the GPU has room for blocks, a row is spread over more threads, one vector each, since
// then only the latency of one row counts.
// Measured: 32768 x 4096 bf16 with a residual, r and e4m3 in groups of 128 165 us, 5.7 TB/s (0.86 of a copy's rate);
// 8192 x 2048 bf16 with r and y 19 us; 16 x 4096 to e4m3 2.9 us.
#include <cuda_fp8.h>

#include "norm.cuh"

namespace gdr {
namespace layer {
namespace {

// Columns [c, c + 8) of a row of y8; word: they start on an 8-byte boundary (CUT: or on a 4-byte one).
template <bool CUT>
__device__ __forceinline__ void store_e4m3(uint8_t* row, const float (&y)[8], float inv, int c, int D, bool word) {
    __nv_fp8x2_storage_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        q[i] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * i] * inv, y[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    uint8_t* p = row + c;
    if (word && (!CUT || c >= 0) && c + 8 <= D) {
        const uint32_t lo = (uint32_t)q[0] | (uint32_t)q[1] << 16, hi = (uint32_t)q[2] | (uint32_t)q[3] << 16;
        if (!CUT || (reinterpret_cast<uintptr_t>(p) & 7) == 0) {
            *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
        } else {
            reinterpret_cast<uint32_t*>(p)[0] = lo;
            reinterpret_cast<uint32_t*>(p)[1] = hi;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i >= 0 && c + i < D) p[i] = (uint8_t)(q[i >> 1] >> (8 * (i & 1)));
    }
}

// CUT: rows cut at 16-byte boundaries, see load_cut.
template <typename IO, int TPR, int VPT, bool CUT>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR, blocks_per_sm<TPR, VPT>())
norm_forward_kernel(NormArgs a, RowTensor x, RowTensor res, const IO* __restrict__ w, IO* __restrict__ y,
                    IO* __restrict__ r, uint8_t* __restrict__ y8, float* __restrict__ scales, bool vec_w, bool vec_y,
                    bool vec_r, bool vec_8) {
    constexpr int RPB = TPR < 128 ? 128 / TPR : 1;
    __shared__ float red[2 * 32], redm[2 * 32];
    extern __shared__ int tops[];             // CUT, groups: [2][RPB][groups], a row's largest |y| of each group
    const int tid = threadIdx.x % TPR, slot = threadIdx.x / TPR;
    const int D = a.D;
    const int shift = CUT ? first_shift<IO>((int64_t)blockIdx.x * RPB + slot, D) : 0;
    Raw8<IO> wr[VPT], xr[VPT], sr[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (tid + i * TPR) * 8 - shift;
        wr[i] = CUT ? load_cut(w, c, D, vec_w && shift == 0) : load8(w + c, D - c, vec_w);
    }
    const bool two = res.p != nullptr;
    const auto fetch = [&](int64_t row) {     // a block's last rows may not exist: zeros
        const IO* xp = reinterpret_cast<const IO*>(x.p) + row * x.ld;
        const IO* sp = reinterpret_cast<const IO*>(res.p) + row * res.ld;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * TPR) * 8 - shift, left = row < a.rows ? D - c : 0;
            if (CUT) {
                xr[i] = load_around(reinterpret_cast<const IO*>(x.p), left > 0 ? row * D + c : 0, a.rows * D);
                if (two) sr[i] = load_around(reinterpret_cast<const IO*>(res.p), left > 0 ? row * D + c : 0, a.rows * D);
            } else {                 // rows that start anywhere by elements: 16384 x 4096 at a stride of 4097 to e4m3 121 us
                                     // bf16, 150 fp32; from the aligned blocks around a vector 127 and 165
                xr[i] = load8(xp + c, left, x.vec);
                if (two) sr[i] = load8(sp + c, left, res.vec);
            }
        }
    };
    fetch((int64_t)blockIdx.x * RPB + slot);
    const int groups = y8 && a.group ? (D + a.group - 1) / a.group : 0;
    if (CUT)
        for (int g = tid; g < groups; g += TPR) tops[slot * groups + g] = 0;
    int turn = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < a.rows; row0 += (int64_t)gridDim.x * RPB, ++turn) {
        const int64_t row = row0 + slot;
        const bool live = row < a.rows;       // threads of a row that does not exist stay for the shuffles
        float v[VPT][8], sum[1] = {0.f};
        if (CUT)
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = (tid + i * TPR) * 8 - shift;
                mask_cut(xr[i], c, D);
                if (two) mask_cut(sr[i], c, D);
                if (live && c < D && ends_past(row, a.rows, c, D)) {
                    xr[i] = load_cut(reinterpret_cast<const IO*>(x.p) + row * D, c, D, false);
                    if (two) sr[i] = load_cut(reinterpret_cast<const IO*>(res.p) + row * D, c, D, false);
                }
            }
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
            const int c = (tid + i * TPR) * 8 - shift;
            if (CUT) {
                if (r && live) store_cut(r + row * D, v[i], c, D, vec_r);
            } else if (r) {
                store_n(r + row * D + c, v[i], live ? D - c : 0, vec_r);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[0] = fmaf(v[i][j], v[i][j], sum[0]);
        }
        row_reduce<TPR, 1, false>(sum, red, turn);
        if (CUT) {                               // the row before has been read out
            if (TPR == 32) __syncwarp();
            for (int g = tid; g < groups; g += TPR) tops[((turn + 1 & 1) * RPB + slot) * groups + g] = 0;
        }
        const float rstd = rsqrtf(sum[0] / (float)D + a.eps);
        float top[1] = {0.f};
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * TPR) * 8 - shift;
            float wf[8], m = 0.f;
            widen(wr[i], wf);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] = v[i][j] * rstd * wf[j];
                if (y8) m = max_nan(m, fabsf(v[i][j]));  // zero past the row's end, or NaN in a row of nothing else
            }
            if (CUT) {
                if (y && live) store_cut(y + row * D, v[i], c, D, vec_y);
            } else if (y) {
                store_n(y + row * D + c, v[i], live ? D - c : 0, vec_y);
            }
            if (CUT && groups) {             // a vector has columns of at most two groups
                int* top = tops + ((turn & 1) * RPB + slot) * groups;
                const int g = max(c, 0) / a.group, next = (g + 1) * a.group - c;
                float lo = 0.f, hi = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < next) lo = max_nan(lo, fabsf(v[i][j]));
                    else hi = max_nan(hi, fabsf(v[i][j]));
                if (c < D) {                 // not negative or NaN: in the order of their bits
                    atomicMax(top + g, __float_as_int(lo));
                    if (next < 8 && c + next < D) atomicMax(top + g + 1, __float_as_int(hi));
                }
            } else if (y8 && a.group) {      // a group's columns lie in group / 8 neighbouring threads
                for (int o = a.group / 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                const float scale = max_nan(m * (1.f / 448.f), 1.17549435e-38f);
                if (live && c < D) {
                    store_e4m3<CUT>(y8 + row * D, v[i], 1.f / scale, c, D, vec_8);
                    if ((c & (a.group - 1)) == 0)
                        scales[row * ((D + a.group - 1) / a.group) + c / a.group] = scale;
                }
            }
            top[0] = max_nan(top[0], m);
        }
        if (CUT && groups) {
            if (TPR == 32) __syncwarp();
            else __syncthreads();
            const int* top = tops + ((turn & 1) * RPB + slot) * groups;
            const auto scale_of = [&](int g) {
                return max_nan(__int_as_float(top[g]) * (1.f / 448.f), 1.17549435e-38f);
            };
            if (live) {
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const int c = (tid + i * TPR) * 8 - shift, g = max(c, 0) / a.group, next = (g + 1) * a.group - c;
                    if (c >= D) continue;
                    const float lo = 1.f / scale_of(g), hi = next < 8 && c + next < D ? 1.f / scale_of(g + 1) : lo;
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i][j] *= j < next ? lo : hi;
                    store_e4m3<CUT>(y8 + row * D, v[i], 1.f, c, D, vec_8);
                }
                for (int g = tid; g < groups; g += TPR) scales[row * groups + g] = scale_of(g);
            }
        }
        if (y8 && !a.group) {
            row_reduce<TPR, 1, true>(top, redm, turn);
            const float scale = max_nan(top[0] * (1.f / 448.f), 1.17549435e-38f), inv = 1.f / scale;
            if (live) {
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const int c = (tid + i * TPR) * 8 - shift;
                    store_e4m3<CUT>(y8 + row * D, v[i], inv, c, D, vec_8);
                }
                if (tid == 0) scales[row] = scale;
            }
        }
    }
}

// Threads of a row and vectors a thread.  Many rows: few threads with two vectors each (up to 4 in the shortest and the
// longest rows), the fewest that hold a row, since what the blocks of an SM have in flight is what counts: 25241 x 2136
// fp16 to e4m3 take 86 us on 160 threads, 102 on 192.  Few rows (less than two blocks an SM): one vector each, as far as a
// block reaches.
Shape shape_of(const NormArgs& a) {
    const int v = vectors_of(a);
    if (v <= 32) return {32, 1};
    const bool few = a.rows < 2 * kSms;
    if (!few && v <= 64) return {32, 2};
    if (!few && v <= 128) return {32, 4};
    if (few)
        for (int tpr = 128; tpr <= 1024; tpr *= 2)
            if (v <= tpr) return {tpr, 1};
    if (v <= 256) return {128, 2};
    if (v <= 320) return {160, 2};
    if (v <= 384) return {192, 2};
    if (v <= 512) return {256, 2};
    if (v <= 768) return {384, 2};
    return {v <= 1024 ? 256 : v <= 2048 ? 512 : 1024, 4};
}

template <typename IO, int TPR, int VPT>
cudaError_t launch_forward(const NormArgs& a, RowTensor x, RowTensor res, const void* w, void* y, void* r, void* y8,
                           float* scales, cudaStream_t s) {
    constexpr int RPB = TPR < 128 ? 128 / TPR : 1, NT = TPR < 128 ? 128 : TPR;
    const int64_t blocks = (a.rows + RPB - 1) / RPB;
    // a wave is a multiple of 8 blocks: of every period of a row's shift
    static_assert(kSms % 8 == 0, "a multiple of the shifts' period");
    const int grid = (int)std::min<int64_t>(blocks, (int64_t)kSms * blocks_per_sm<TPR, VPT>());
    // Cut at the boundaries: rows not aligned, every tensor contiguous from a boundary on.
    bool cut = (int64_t)a.D * sizeof(IO) % 16 != 0 && vectors_of(a) <= TPR * VPT && a.rows * a.D >= 8 && x.ld == a.D &&
               (!res.p || res.ld == a.D);
    for (const void* p : {x.p, res.p, (const void*)y, (const void*)r, (const void*)y8})
        cut = cut && reinterpret_cast<uintptr_t>(p) % 16 == 0;
    const auto al = [&](const void* p, int unit) {
        return (reinterpret_cast<uintptr_t>(p) % 16) == 0 && ((int64_t)a.D * unit) % 16 == 0;
    };
    const auto go = [&](auto in_cuts) {
        constexpr bool kCut = decltype(in_cuts)::value;
        const int bytes = kCut && y8 && a.group ? 2 * RPB * ((a.D + a.group - 1) / a.group) * 4 : 0;
        norm_forward_kernel<IO, TPR, VPT, kCut><<<grid, NT, bytes, s>>>(
            a, x, res, (const IO*)w, (IO*)y, (IO*)r, (uint8_t*)y8, scales, reinterpret_cast<uintptr_t>(w) % 16 == 0,
            cut || al(y, sizeof(IO)), cut || al(r, sizeof(IO)),
            reinterpret_cast<uintptr_t>(y8) % 8 == 0 && (cut || a.D % 8 == 0));
    };
    if constexpr (VPT > 1 || TPR == 32)     // one vector on many threads: few rows, where latency counts
        if (cut) {
            go(std::true_type());
            return cudaGetLastError();
        }
    cut = false;
    go(std::false_type());
    return cudaGetLastError();
}

// Calls f with the shape's constants.
template <typename F> cudaError_t with_shape(Shape h, F f) {
#define GDR_SHAPE(T, V) \
    if (h.tpr == T && h.vpt == V) return f(std::integral_constant<int, T>(), std::integral_constant<int, V>());
    GDR_SHAPE(32, 1) GDR_SHAPE(32, 2) GDR_SHAPE(32, 4)
    GDR_SHAPE(128, 1) GDR_SHAPE(256, 1) GDR_SHAPE(512, 1) GDR_SHAPE(1024, 1)
    GDR_SHAPE(128, 2) GDR_SHAPE(160, 2) GDR_SHAPE(192, 2) GDR_SHAPE(256, 2) GDR_SHAPE(384, 2)
    GDR_SHAPE(256, 4) GDR_SHAPE(512, 4) GDR_SHAPE(1024, 4)
#undef GDR_SHAPE
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t norm_forward(const NormArgs& a, RowTensor x, RowTensor res, const void* w, void* y, void* r, void* y8,
                         float* scales, cudaStream_t s) {
    return with_shape(shape_of(a), [&](auto tpr, auto vpt) {
        constexpr int T = decltype(tpr)::value, V = decltype(vpt)::value;
        if (a.io == GDR_F32) return launch_forward<float, T, V>(a, x, res, w, y, r, y8, scales, s);
        if (a.io == GDR_BF16) return launch_forward<__nv_bfloat16, T, V>(a, x, res, w, y, r, y8, scales, s);
        return launch_forward<__half, T, V>(a, x, res, w, y, r, y8, scales, s);
    });
}

}  // namespace layer
}  // namespace gdr
