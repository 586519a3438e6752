// The gradient of the root-mean-square norm, and the column sums that the layer operators' gradients end in.
//
// With xh = s rstd and the sum taken over the row:
//   ds = rstd (w dy - xh mean(w dy xh)) + dr,   dw = sum over rows of dy xh
// One pass over dy and r: both sums of a row come from registers.  Each block adds its rows' dw in registers and
// leaves one row of partial sums, which column_sum adds in a fixed order: no atomics, the same bits in every run.
// Bound: memory.  Measured: 8192 x 2048 bf16 with dr 25 us, 5.4 TB/s (0.80 of a copy's rate), and 3 us for column_sum;
// 4452 x 4096 fp32 49 us, 6.0 TB/s.  Rows above 4096 columns fit no ring: one block of 256 threads an SM and nothing under
// way but a row's own loads, 4096 x 8192 bf16 with column_sum 74 us, 3.6 TB/s.
#include "norm.cuh"

namespace gdr {
namespace layer {
namespace {

// The backward's rows: dy, r and dr of the next RING - 1 rows of a block are on their way into shared memory, each
// thread's vectors in its own places, while the block works on one.  (With one row ahead in registers, as the forward
// has it, the kernel took twice the time; the forward's two tensors are faster that way, 20 against 28 us at 8192 x
// 2048.)  RING = 1: a row is loaded when it is its turn (few rows, rows not aligned, or rows too wide for the ring).
template <int NT> constexpr int kRingBytes = NT < 512 ? 56 * 1024 : 200 * 1024;   // of a block: several fit an SM, or one
template <typename IO, int NT, int VPT> constexpr int ring_of() {
    constexpr int row = NT * VPT * 3 * (int)sizeof(Raw8<IO>);
    return 4 * row <= kRingBytes<NT> ? 4 : 3 * row <= kRingBytes<NT> ? 3 : 2 * row <= kRingBytes<NT> ? 2 : 1;
}

template <typename IO, int NT, int VPT, int RING, bool CUT> struct Pipe {
    const IO* base[3];            // the tensors, or nullptr
    int64_t rows;
    int D, tid, tpr, shift;
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
                        const int c = (tid + i * tpr) * 8 - shift;
                        if (c < D && !(CUT && ends_past(row, rows, c, D))) {
#pragma unroll
                            for (int part = 0; part < (int)sizeof(IO) / 2; ++part)
                                copy_ahead(reinterpret_cast<RawN<IO, 16 / sizeof(IO)>*>(place(slot, t, i, part)),
                                           base[t] + row * D + c + part * (16 / (int)sizeof(IO)));
                        } else if (CUT && c < D) {
                            const Raw8<IO> v = load_cut(base[t] + row * D, c, D, false);
#pragma unroll
                            for (int part = 0; part < (int)sizeof(IO) / 2; ++part)
                                *place(slot, t, i, part) = reinterpret_cast<const uint4*>(&v)[part];
                        }
                    }
        copy_group();
    }
    // The thread's vectors of tensor t of the row; zeros past the row's end and for a row that does not exist.  Without a ring
    // nothing but a row's own loads is under way, so none may wait for another: with load_cut, whose element by element branch
    // fills the registers of 16-bit vectors in halves, each did (4096 x 5120 bf16 131 us, 68 so; 8192 x 4095 291 and 185).
    // Rows that start anywhere: fp32 vectors come from the blocks around them (4452 x 4096 115 us, 123 by elements), 16-bit
    // ones by elements (8192 x 2048 66 us, 72 from blocks).
    __device__ __forceinline__ void take(int64_t row, int slot, int t, Raw8<IO> (&v)[VPT]) const {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * tpr) * 8 - shift, left = row < rows ? D - c : 0;
            if (RING == 1 && CUT) {
                v[i] = load_around(base[t], left > 0 ? row * D + c : 0, rows * D);
            } else if (RING == 1) {
                v[i] = load8(base[t] + row * D + c, left, vec, sizeof(IO) == 4 ? c : 0);
            } else if (left > 0) {
#pragma unroll
                for (int part = 0; part < (int)sizeof(IO) / 2; ++part)
                    reinterpret_cast<uint4*>(&v[i])[part] = *place(slot, t, i, part);
                if (CUT) mask_cut(v[i], c, D);
            } else {
                v[i] = load8((const IO*)nullptr, 0, false);
            }
        }
        if (RING == 1 && CUT)          // when all loads are under way: see load_around
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = (tid + i * tpr) * 8 - shift;
                mask_cut(v[i], c, row < rows ? D : 0);
                if (row < rows && c < D && ends_past(row, rows, c, D)) v[i] = load_cut(base[t] + row * D, c, D, false);
            }
    }
};

template <typename IO, int TPR, int VPT, int RING, bool CUT>
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
    const int shift = CUT ? first_shift<IO>((int64_t)blockIdx.x * RPB + slot, D) : 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        wr[i] = load_cut(w, (tid + i * TPR) * 8 - shift, D, vec && shift == 0);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
    }
    const int64_t step = (int64_t)gridDim.x * RPB, first = (int64_t)blockIdx.x * RPB + slot;
    const Pipe<IO, NT, VPT, RING, CUT> in{{dy, r, dr}, a.rows, D, tid, TPR, shift, vec, smem};
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
            const int c = (tid + i * TPR) * 8 - shift;
            float s[8], g[8], wf[8], o[8];
            widen(rr[i], s), widen(yr[i], g), widen(wr[i], wf);
            if (dr) widen(er[i], o);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                o[j] = fmaf(rstd, fmaf(-s[j], back, wf[j] * g[j]), dr ? o[j] : 0.f);
                if (live) dw[i][j] = fmaf(g[j], s[j] * rstd, dw[i][j]);
            }
            if (CUT) {
                if (live) store_cut(dx + row * D, o, c, D, vec);
            } else if (live) {
                store_n(dx + row * D + c, o, D - c, vec);
            }
        }
    }
    float* mine = partial + ((int64_t)blockIdx.x * RPB + slot) * D;
#pragma unroll
    for (int i = 0; i < VPT; ++i) store_cut(mine, dw[i], (tid + i * TPR) * 8 - shift, D, (D & 3) == 0 && shift == 0);
}

// 32 columns a block, 32 rows in flight; the 32 partial sums of a column are added in shared memory in order.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* __restrict__ in, int64_t rows, int64_t ld,
                                                          int64_t cols, float* __restrict__ out, int64_t cols2,
                                                          float* __restrict__ out2) {
    __shared__ float part[32][33];
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    asm volatile("griddepcontrol.wait;" ::: "memory");      // the kernel before is done
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

// The gradient's: one vector a thread as far as 512 threads reach, since its sums of dw and a row's inputs fill the
// registers at two (30 us instead of 25 at 8192 x 2048 bf16; 77 instead of 49 on 512 threads at 4452 x 4096 fp32).
Shape backward_shape(const NormArgs& a) {
    const int v = vectors_of(a);
    if (v <= 64) return {32, v <= 32 ? 1 : 2};
    if (v <= 256) return {v <= 128 ? 128 : 256, 1};
    if (v <= 512) return {512, 1};
    return {v <= 1024 ? 256 : v <= 2048 ? 512 : 1024, 4};
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
    bool vec = true;
    for (const void* p : {dy, r, w, dr, (const void*)dx}) vec = vec && reinterpret_cast<uintptr_t>(p) % 16 == 0;
    const bool odd = (int64_t)a.D * sizeof(IO) % 16 != 0;           // rows not aligned: cut at the boundaries
    const bool cut = vec && odd && vectors_of(a) <= TPR * VPT && a.rows * a.D >= 8;
    vec = vec && (cut || !odd);
    const int64_t grid = backward_grid(a, {TPR, VPT});
    const auto go = [&](auto ring, auto in_cuts) {
        constexpr int R = decltype(ring)::value, bytes = R > 1 ? R * NT * VPT * 3 * (int)sizeof(Raw8<IO>) : 0;
        const auto kernel = norm_backward_kernel<IO, TPR, VPT, R, decltype(in_cuts)::value>;
        if (bytes > 40 * 1024)
            if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) return e;
        kernel<<<(unsigned)grid, NT, bytes, s>>>(a, (const IO*)dy, (const IO*)r, (const IO*)w, (const IO*)dr, (IO*)dx,
                                                 partial, vec);
        return cudaGetLastError();
    };
    const bool turns = RING > 1 && vec && grid * RPB < a.rows;
    if (cut) return turns ? go(std::integral_constant<int, RING>(), std::true_type())
                          : go(std::integral_constant<int, 1>(), std::true_type());
    if (turns && a.D % 8 == 0) return go(std::integral_constant<int, RING>(), std::false_type());
    return go(std::integral_constant<int, 1>(), std::false_type());
}

// Calls f with the shape's constants.
template <typename F> cudaError_t with_shape(Shape h, F f) {
#define GDR_SHAPE(T, V) \
    if (h.tpr == T && h.vpt == V) return f(std::integral_constant<int, T>(), std::integral_constant<int, V>());
    GDR_SHAPE(32, 1) GDR_SHAPE(32, 2) GDR_SHAPE(128, 1) GDR_SHAPE(256, 1) GDR_SHAPE(512, 1)
    GDR_SHAPE(256, 4) GDR_SHAPE(512, 4) GDR_SHAPE(1024, 4)
#undef GDR_SHAPE
    return cudaErrorInvalidValue;
}

}  // namespace

int64_t norm_partial_rows(const NormArgs& a) {
    const Shape h = backward_shape(a);
    return backward_grid(a, h) * (h.tpr < 128 ? 128 / h.tpr : 1);
}

cudaError_t norm_backward(const NormArgs& a, const void* dy, const void* r, const void* w, const void* dr, void* dx,
                          float* dw, float* partial, cudaStream_t s) {
    const cudaError_t e = with_shape(backward_shape(a), [&](auto tpr, auto vpt) {
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
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config{};
    config.gridDim = dim3((unsigned)((cols + cols2 + 31) / 32));
    config.blockDim = dim3(32, 32);
    config.stream = s;
    config.attrs = &early;
    config.numAttrs = 1;
    return cudaLaunchKernelEx(&config, column_sum_kernel, in, rows, ld, cols, out, cols2, out2);
}

}  // namespace layer
}  // namespace gdr
