// The layer norm of a row with the residual's addition, and its gradient.
//
//   s = x + residual, m = mean s, rstd = 1 / sqrt(mean (s - m)^2 + eps), y = (s - m) rstd w + b   (fp32, rounded once)
//   xh = (s - m) rstd,  ds = rstd (w dy - mean(w dy) - xh mean(w dy xh)) + dr,  dw = sum dy xh,  db = sum dy
//
// Bound: memory.  A row is read once and stays in registers between its two sums (the mean first, then the squares around
// it: one pass over squares would lose a row whose mean is far from zero) and the output.
#include "norm.cuh"

namespace gdr {
namespace layer {
namespace {

template <typename IO, int TPR, int VPT>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
layernorm_forward_kernel(NormArgs a, RowTensor x, RowTensor res, const IO* __restrict__ w, const IO* __restrict__ b,
                         IO* __restrict__ y, IO* __restrict__ r, bool vec_w, bool vec_y) {
    constexpr int RPB = TPR < 128 ? 128 / TPR : 1;
    __shared__ float red[2][2 * 32];
    const int tid = threadIdx.x % TPR, slot = threadIdx.x / TPR, D = a.D;
    int turn = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < a.rows; row0 += (int64_t)gridDim.x * RPB, ++turn) {
        const int64_t row = row0 + slot;
        const bool live = row < a.rows;       // threads of a row that does not exist stay for the shuffles
        float v[VPT][8], sum[1] = {0.f}, var[1] = {0.f};
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * TPR) * 8, left = live ? D - c : 0;
            widen(load8((const IO*)x.p + row * x.ld + c, left, x.vec, c), v[i]);
            if (res.p) {
                float t[8];
                widen(load8((const IO*)res.p + row * res.ld + c, left, res.vec, c), t);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += t[j];
            }
            if (r) store_n(r + row * D + c, v[i], left, vec_y);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[0] += v[i][j];
        }
        row_reduce<TPR, 1, false>(sum, red[0], turn);
        const float mean = sum[0] / (float)D;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * TPR) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] = c + j < D ? v[i][j] - mean : 0.f;
                var[0] = fmaf(v[i][j], v[i][j], var[0]);
            }
        }
        row_reduce<TPR, 1, false>(var, red[1], turn);
        const float rstd = rsqrtf(var[0] / (float)D + a.eps);
        if (!y) continue;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * TPR) * 8;
            float wf[8], bf[8];
            widen(load8(w + c, D - c, vec_w, c), wf);
            widen(load8(b + c, b ? D - c : 0, vec_w, c), bf);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = fmaf(v[i][j] * rstd, wf[j], bf[j]);
            store_n(y + row * D + c, v[i], live ? D - c : 0, vec_y);
        }
    }
}

template <typename IO, int TPR, int VPT>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
layernorm_backward_kernel(NormArgs a, const IO* __restrict__ dy, const IO* __restrict__ r, const IO* __restrict__ w,
                          const IO* __restrict__ dr, IO* __restrict__ dx, float* __restrict__ partial, bool vec) {
    constexpr int RPB = TPR < 128 ? 128 / TPR : 1;
    __shared__ float red[2][2 * 2 * 32];
    const int tid = threadIdx.x % TPR, slot = threadIdx.x / TPR, D = a.D;
    float dw[VPT][8], db[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = db[i][j] = 0.f;
    int turn = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < a.rows; row0 += (int64_t)gridDim.x * RPB, ++turn) {
        const int64_t row = row0 + slot;
        const bool live = row < a.rows;
        float s[VPT][8], g[VPT][8], one[2] = {0.f, 0.f}, two[2] = {0.f, 0.f};
        Raw8<IO> wr[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * TPR) * 8, left = live ? D - c : 0;
            float wf[8];
            widen(load8(r + row * D + c, left, vec, c), s[i]);
            widen(load8(dy + row * D + c, left, vec, c), g[i]);
            wr[i] = load8(w + c, D - c, vec, c);
            widen(wr[i], wf);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                one[0] += s[i][j];
                one[1] = fmaf(wf[j], g[i][j], one[1]);
            }
        }
        row_reduce<TPR, 2, false>(one, red[0], turn);
        const float mean = one[0] / (float)D, flat = one[1] / (float)D;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * TPR) * 8;
            float wf[8];
            widen(wr[i], wf);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s[i][j] = c + j < D ? s[i][j] - mean : 0.f;
                two[0] = fmaf(s[i][j], s[i][j], two[0]);
                two[1] = fmaf(wf[j] * g[i][j], s[i][j], two[1]);
            }
        }
        row_reduce<TPR, 2, false>(two, red[1], turn);
        const float rstd = rsqrtf(two[0] / (float)D + a.eps), back = two[1] / (float)D * rstd * rstd;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * TPR) * 8;
            float wf[8], o[8];
            widen(wr[i], wf);
            widen(load8(dr + row * D + c, live && dr ? D - c : 0, vec, c), o);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                o[j] = fmaf(rstd, fmaf(-s[i][j], back, fmaf(wf[j], g[i][j], -flat)), o[j]);
                if (live) dw[i][j] = fmaf(g[i][j], s[i][j] * rstd, dw[i][j]), db[i][j] += g[i][j];
            }
            store_n(dx + row * D + c, o, live ? D - c : 0, vec);
        }
    }
    float* mine = partial + ((int64_t)blockIdx.x * RPB + slot) * 2 * D;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        store_cut(mine, dw[i], (tid + i * TPR) * 8, D, (D & 3) == 0);
        store_cut(mine + D, db[i], (tid + i * TPR) * 8, D, (D & 3) == 0);
    }
}

Shape shape_of(int D) {
    const int v = (D + 7) / 8;
    if (v <= 64) return {32, v <= 32 ? 1 : 2};
    if (v <= 128) return {128, 1};
    if (v <= 256) return {256, 1};
    if (v <= 512) return {512, 1};
    return {v <= 1024 ? 256 : v <= 2048 ? 512 : 1024, 4};
}

int64_t grid_of(const NormArgs& a, Shape h) {
    const int rpb = h.tpr < 128 ? 128 / h.tpr : 1, nt = h.tpr < 128 ? 128 : h.tpr;
    return std::min<int64_t>((a.rows + rpb - 1) / rpb, (int64_t)kSms * std::max(1, (h.vpt > 2 ? 512 : 1024) / nt));
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

template <typename F> cudaError_t with_types(int io, Shape h, F f) {
    return with_shape(h, [&](auto t, auto v) {
        if (io == GDR_F32) return f(float(), t, v);
        if (io == GDR_BF16) return f(__nv_bfloat16(), t, v);
        return f(__half(), t, v);
    });
}

bool on_16(std::initializer_list<const void*> ps, int64_t row_bytes) {
    bool vec = row_bytes % 16 == 0;
    for (const void* p : ps) vec = vec && reinterpret_cast<uintptr_t>(p) % 16 == 0;
    return vec;
}

}  // namespace

cudaError_t layernorm_forward(const NormArgs& a, RowTensor x, RowTensor res, const void* w, const void* b, void* y,
                              void* r, cudaStream_t s) {
    const Shape h = shape_of(a.D);
    return with_types(a.io, h, [&](auto io, auto tpr, auto vpt) {
        using IO = decltype(io);
        constexpr int T = decltype(tpr)::value, V = decltype(vpt)::value;
        layernorm_forward_kernel<IO, T, V><<<(unsigned)grid_of(a, h), T < 128 ? 128 : T, 0, s>>>(
            a, x, res, (const IO*)w, (const IO*)b, (IO*)y, (IO*)r, on_16({w, b}, 16),
            on_16({y, r}, (int64_t)a.D * sizeof(IO)));
        return cudaGetLastError();
    });
}

int64_t layernorm_partial_rows(const NormArgs& a) {
    const Shape h = shape_of(a.D);
    return grid_of(a, h) * (h.tpr < 128 ? 128 / h.tpr : 1);
}

cudaError_t layernorm_backward(const NormArgs& a, const void* dy, const void* r, const void* w, const void* dr, void* dx,
                               float* dw, float* db, float* partial, cudaStream_t s) {
    const Shape h = shape_of(a.D);
    const cudaError_t e = with_types(a.io, h, [&](auto io, auto tpr, auto vpt) {
        using IO = decltype(io);
        constexpr int T = decltype(tpr)::value, V = decltype(vpt)::value;
        layernorm_backward_kernel<IO, T, V><<<(unsigned)grid_of(a, h), T < 128 ? 128 : T, 0, s>>>(
            a, (const IO*)dy, (const IO*)r, (const IO*)w, (const IO*)dr, (IO*)dx, partial,
            on_16({dy, r, w, dr, dx}, (int64_t)a.D * sizeof(IO)));
        return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
    return column_sum(partial, layernorm_partial_rows(a), 2 * (int64_t)a.D, a.D, dw, a.D, db, s);
}

}  // namespace layer
}  // namespace gdr
