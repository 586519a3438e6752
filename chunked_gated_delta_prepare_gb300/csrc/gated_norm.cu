// The gated norm of a recurrence's output, a row of V columns being one head of one token, and its gradient.
//
//   n = x rstd, rstd = 1 / sqrt(mean x^2 + eps),  y = n w f(z),  f = silu or sigmoid
//   dn = dy w f(z),  dx = rstd (dn - n mean(dn n)),  dz = dy n w f'(z),  dw = sum dy n f(z)
//
// Bound: memory.  A row lies on TPR threads (4 to 32 up to 1024 columns, sums by shuffles; a block above), and a row's place
// in the grid keeps its head: the number of places is a multiple of H, so w and the sums of dw stay in registers.
#include "norm.cuh"

namespace gdr {
namespace layer {
namespace {

constexpr int kThreads = 256;

struct Places {              // of rows in the grid: place p has head p % H of the tokens p / H + k * step
    int64_t count, step, turns;
};

// Sums over a row's TPR lanes, or the block.
template <int TPR> __device__ __forceinline__ void sum_row(float (&v)[1], float* red, int turn) {
    if constexpr (TPR >= 32) {
        row_reduce<TPR, 1, false>(v, red, turn);
    } else {
#pragma unroll
        for (int o = TPR / 2; o > 0; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    }
}

// f(z) and its slope.
template <bool SILU> __device__ __forceinline__ float gate_of(float z) { return SILU ? z * sigmoid(z) : sigmoid(z); }
template <bool SILU> __device__ __forceinline__ float2 gate_and_slope(float z) {
    // with e = e^-|z| <= 1 both sigmoid(z) and 1 - sigmoid(z) keep their relative accuracy
    const float e = ex2(-fabsf(z) * kLog2e), p = rcp(1.f + e), q = e * p;
    const float s = z < 0.f ? q : p, rest = z < 0.f ? p : q;
    return SILU ? make_float2(z * s, s * fmaf(z, rest, 1.f)) : make_float2(s, s * rest);
}

template <typename IO, int TPR, int VPT, bool SILU>
__global__ void __launch_bounds__(TPR > kThreads ? TPR : kThreads)
gated_norm_forward_kernel(GatedNormArgs a, Places pl, RowTensor x, RowTensor z, const IO* __restrict__ w,
                          IO* __restrict__ y, bool vec_w, bool vec_y) {
    constexpr int NT = TPR > kThreads ? TPR : kThreads, RPB = NT / TPR;
    __shared__ float red[2 * 32];
    const int tid = threadIdx.x % TPR, V = a.V;
    const int64_t place = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    const int head = (int)(place % a.H);
    const int64_t token0 = place / a.H;
    const IO* wp = w + (a.per_head ? (int64_t)head * V : 0);
    for (int64_t turn = 0; turn < pl.turns; ++turn) {
        const int64_t token = token0 + turn * pl.step;
        const bool live = place < pl.count && token < a.tokens;
        float v[VPT][8], sum[1] = {0.f};
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * TPR) * 8;
            widen(load8((const IO*)x.p + token * x.ld + (int64_t)head * V + c, live ? V - c : 0, x.vec, c), v[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[0] = fmaf(v[i][j], v[i][j], sum[0]);
        }
        sum_row<TPR>(sum, red, (int)turn);
        const float rstd = rsqrtf(sum[0] / (float)V + a.eps);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * TPR) * 8;
            float zf[8], wf[8];
            widen(load8((const IO*)z.p + token * z.ld + (int64_t)head * V + c, live ? V - c : 0, z.vec, c), zf);
            widen(load8(wp + c, V - c, vec_w, c), wf);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * wf[j] * gate_of<SILU>(zf[j]);
            store_n(y + (token * a.H + head) * V + c, v[i], live ? V - c : 0, vec_y);
        }
    }
}

// partial: a row of V sums for each place.
template <typename IO, int TPR, int VPT, bool SILU>
__global__ void __launch_bounds__(TPR > kThreads ? TPR : kThreads)
gated_norm_backward_kernel(GatedNormArgs a, Places pl, const IO* __restrict__ dy, RowTensor x, RowTensor z,
                           const IO* __restrict__ w, IO* __restrict__ dx, IO* __restrict__ dz,
                           float* __restrict__ partial, bool vec_w, bool vec) {
    constexpr int NT = TPR > kThreads ? TPR : kThreads, RPB = NT / TPR;
    __shared__ float red[2][2 * 32];
    const int tid = threadIdx.x % TPR, V = a.V;
    const int64_t place = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    const int head = (int)(place % a.H);
    const int64_t token0 = place / a.H;
    const IO* wp = w + (a.per_head ? (int64_t)head * V : 0);
    float dw[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
    for (int64_t turn = 0; turn < pl.turns; ++turn) {
        const int64_t token = token0 + turn * pl.step;
        const bool live = place < pl.count && token < a.tokens;
        Raw8<IO> xr[VPT], zr[VPT], gr[VPT], wr[VPT];
        float sq[1] = {0.f}, dot[1] = {0.f};
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * TPR) * 8, left = live ? V - c : 0;
            const int64_t at = (token * a.H + head) * V + c;
            xr[i] = load8((const IO*)x.p + token * x.ld + (int64_t)head * V + c, left, x.vec, c);
            zr[i] = load8((const IO*)z.p + token * z.ld + (int64_t)head * V + c, left, z.vec, c);
            gr[i] = load8(dy + at, left, vec, c);
            wr[i] = load8(wp + c, V - c, vec_w, c);
            float xf[8], zf[8], gf[8], wf[8];
            widen(xr[i], xf), widen(zr[i], zf), widen(gr[i], gf), widen(wr[i], wf);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sq[0] = fmaf(xf[j], xf[j], sq[0]);
                dot[0] = fmaf(gf[j] * wf[j] * gate_of<SILU>(zf[j]), xf[j], dot[0]);
            }
        }
        sum_row<TPR>(sq, red[0], (int)turn);
        sum_row<TPR>(dot, red[1], (int)turn);
        const float rstd = rsqrtf(sq[0] / (float)V + a.eps), back = dot[0] / (float)V * rstd * rstd;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * TPR) * 8, left = live ? V - c : 0;
            const int64_t at = (token * a.H + head) * V + c;
            float xf[8], zf[8], gf[8], wf[8], o[8], oz[8];
            widen(xr[i], xf), widen(zr[i], zf), widen(gr[i], gf), widen(wr[i], wf);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 f = gate_and_slope<SILU>(zf[j]);
                const float n = xf[j] * rstd, gw = gf[j] * wf[j];
                o[j] = rstd * fmaf(-xf[j], back, gw * f.x);
                oz[j] = gw * n * f.y;
                if (live) dw[i][j] = fmaf(gf[j] * n, f.x, dw[i][j]);
            }
            store_n(dx + at, o, left, vec);
            store_n(dz + at, oz, left, vec);
        }
    }
    if (place < pl.count)
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            store_cut(partial + place * V, dw[i], (tid + i * TPR) * 8, V, (V & 3) == 0);
}

Shape shape_of(int V) {
    const int v = (V + 7) / 8;
    if (v <= 32) return {v <= 4 ? 4 : v <= 8 ? 8 : v <= 16 ? 16 : 32, 1};
    if (v <= 128) return {32, v <= 64 ? 2 : 4};
    return {v <= 512 ? 256 : 512, 2};
}

// Blocks an SM: 4 of 256 threads.
Places places_of(const GatedNormArgs& a, Shape h) {
    const int64_t rpb = std::max(h.tpr, kThreads) / h.tpr, most = (int64_t)kSms * 4 * rpb;
    Places p;
    p.step = std::min<int64_t>(a.tokens, std::max<int64_t>(1, most / a.H));
    p.count = p.step * a.H;
    p.turns = (a.tokens + p.step - 1) / p.step;
    return p;
}

// Calls f with the io type and the shape's constants.
template <typename F> cudaError_t with_types(const GatedNormArgs& a, Shape h, F f) {
    const auto types = [&](auto t, auto v) {
        const auto gates = [&](auto io) {
            return a.silu ? f(io, t, v, std::true_type()) : f(io, t, v, std::false_type());
        };
        if (a.io == GDR_F32) return gates(float());
        if (a.io == GDR_BF16) return gates(__nv_bfloat16());
        return gates(__half());
    };
#define GDR_SHAPE(T, V) \
    if (h.tpr == T && h.vpt == V) return types(std::integral_constant<int, T>(), std::integral_constant<int, V>());
    GDR_SHAPE(4, 1) GDR_SHAPE(8, 1) GDR_SHAPE(16, 1) GDR_SHAPE(32, 1) GDR_SHAPE(32, 2) GDR_SHAPE(32, 4)
    GDR_SHAPE(256, 2) GDR_SHAPE(512, 2)
#undef GDR_SHAPE
    return cudaErrorInvalidValue;
}

// Whether the heads' rows of all these tensors start on 16-byte boundaries.
bool on_16(std::initializer_list<const void*> ps, int64_t head_bytes) {
    bool vec = head_bytes % 16 == 0;
    for (const void* p : ps) vec = vec && reinterpret_cast<uintptr_t>(p) % 16 == 0;
    return vec;
}

}  // namespace

cudaError_t gated_norm_forward(const GatedNormArgs& a, RowTensor x, RowTensor z, const void* w, void* y, cudaStream_t s) {
    const Shape h = shape_of(a.V);
    const Places p = places_of(a, h);
    return with_types(a, h, [&](auto io, auto tpr, auto vpt, auto silu) {
        using IO = decltype(io);
        constexpr int T = decltype(tpr)::value, NT = T > kThreads ? T : kThreads;
        const int64_t bytes = (int64_t)a.V * sizeof(IO);
        x.vec = x.vec && bytes % 16 == 0, z.vec = z.vec && bytes % 16 == 0;
        gated_norm_forward_kernel<IO, T, decltype(vpt)::value, decltype(silu)::value>
            <<<(unsigned)((p.count + NT / T - 1) / (NT / T)), NT, 0, s>>>(a, p, x, z, (const IO*)w, (IO*)y, on_16({w}, bytes),
                                                                        on_16({y}, bytes));
        return cudaGetLastError();
    });
}

int64_t gated_norm_partial_rows(const GatedNormArgs& a) { return places_of(a, shape_of(a.V)).count; }

cudaError_t gated_norm_backward(const GatedNormArgs& a, const void* dy, RowTensor x, RowTensor z, const void* w, void* dx,
                                void* dz, float* dw, float* partial, cudaStream_t s) {
    const Shape h = shape_of(a.V);
    const Places p = places_of(a, h);
    const cudaError_t e = with_types(a, h, [&](auto io, auto tpr, auto vpt, auto silu) {
        using IO = decltype(io);
        constexpr int T = decltype(tpr)::value, NT = T > kThreads ? T : kThreads;
        const int64_t bytes = (int64_t)a.V * sizeof(IO);
        x.vec = x.vec && bytes % 16 == 0, z.vec = z.vec && bytes % 16 == 0;
        gated_norm_backward_kernel<IO, T, decltype(vpt)::value, decltype(silu)::value>
            <<<(unsigned)((p.count + NT / T - 1) / (NT / T)), NT, 0, s>>>(a, p, (const IO*)dy, x, z, (const IO*)w, (IO*)dx,
                                                                        (IO*)dz, partial, on_16({w}, bytes),
                                                                        on_16({dy, dx, dz}, bytes));
        return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
    const int64_t cols = (int64_t)a.V * (a.per_head ? a.H : 1);
    return column_sum(partial, p.count * a.V / cols, cols, cols, dw, 0, nullptr, s);
}

}  // namespace layer
}  // namespace gdr
