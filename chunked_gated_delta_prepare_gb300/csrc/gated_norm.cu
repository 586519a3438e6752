// The gated norm of a recurrence's output, a row of V columns being one head of one token, and its gradient.
//
//   n = x rstd, rstd = 1 / sqrt(mean x^2 + eps),  y = n w f(z),  f = silu or sigmoid
//   dn = dy w f(z),  dx = rstd (dn - n mean(dn n)),  dz = dy n w f'(z),  dw = sum dy n f(z)
//
// Bound: memory.  A row lies on TPR threads (4 to 32 up to 256 columns, sums by shuffles; a block above), and a row's place
// in the grid keeps its head: the number of places is a multiple of H, so w and the sums of dw stay in registers.
//
// Measured (bf16, heads of 128): 32768 x 32 heads in 136 us, 5.9 TB/s, 0.87 of a copy's rate; 8192 x 16 forward 17.5,
// gradient 31, 0.8, and 3 for column_sum.  The same holds for heads of 64 to 2048 columns; wider rows take a block of 512
// threads that has one row in flight (4096 columns: 4.5 TB/s, 8192: 3.7).  Heads of other than whole 16 bytes go by elements
// (100 columns 2.3 TB/s, 33 1.7); vectors cut at the boundaries measured slower (2.0, 1.3).
#include "norm.cuh"

namespace gdr {
namespace layer {
namespace {

constexpr int block_of(int tpr) { return tpr <= 32 ? 256 : tpr; }      // a row of more than a warp is a block's

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

// f(z) of two, and its slope: with e = e^-|z| <= 1 both sigmoid(z) and 1 - sigmoid(z) keep their relative accuracy.
template <bool SILU> __device__ __forceinline__ F2 gate2(F2 z) { return SILU ? silu2(z) : sigmoid2(z); }
template <bool SILU> __device__ __forceinline__ void gate_and_slope2(F2 z, F2& f, F2& slope) {
    const float2 v = unpack2(z);
    const F2 e = pack2(ex2(-fabsf(v.x) * kLog2e), ex2(-fabsf(v.y) * kLog2e));
    const F2 large = rcp_2(add2(both(1.f), e)), small = mul2(e, large);
    const float2 l = unpack2(large), q = unpack2(small);
    const F2 s = pack2(v.x < 0.f ? q.x : l.x, v.y < 0.f ? q.y : l.y);
    const F2 rest = pack2(v.x < 0.f ? l.x : q.x, v.y < 0.f ? l.y : q.y);
    f = SILU ? mul2(z, s) : s;
    slope = SILU ? mul2(s, fma2(z, rest, both(1.f))) : mul2(s, rest);
}
__device__ __forceinline__ float both_halves(F2 v) {
    const float2 f = unpack2(v);
    return f.x + f.y;
}
template <typename IO> __device__ __forceinline__ void store_pairs(IO* p, const F2 (&v)[4], int left, bool vec) {
    float x[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 f = unpack2(v[k]);
        x[2 * k] = f.x, x[2 * k + 1] = f.y;
    }
    store_n(p, x, left, vec);
}

// Blocks an SM that the registers leave room for (64, 128 a thread at one vector); the grid is one wave of them.
constexpr int forward_blocks(int tpr, int vpt) { return (vpt == 1 ? 1024 : 512) / block_of(tpr); }
constexpr int backward_blocks(int tpr, int vpt) { return vpt == 1 ? 512 / block_of(tpr) : 1; }

// Rows of one place that are loaded together: what the threads have in flight is what counts.
template <int VPT> constexpr int kTogether = VPT == 1 ? 2 : 1;

template <typename IO, int TPR, int VPT, bool SILU>
__global__ void __launch_bounds__(block_of(TPR), forward_blocks(TPR, VPT))
gated_norm_forward_kernel(GatedNormArgs a, Places pl, RowTensor x, RowTensor z, const IO* __restrict__ w,
                          IO* __restrict__ y, bool vec_w, bool vec_y) {
    constexpr int NT = block_of(TPR), RPB = NT / TPR, U = kTogether<VPT>;
    __shared__ float red[2 * 32];
    const int tid = threadIdx.x % TPR, V = a.V;
    const int64_t place = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    const int head = (int)(place % a.H);
    const int64_t token0 = place / a.H;
    const IO* wp = w + (a.per_head ? (int64_t)head * V : 0);
    Raw8<IO> wr[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) wr[i] = load8(wp + (tid + i * TPR) * 8, V - (tid + i * TPR) * 8, vec_w, (tid + i * TPR) * 8);
    const float over = 1.f / (float)V;
    for (int64_t turn = 0; turn < pl.turns; turn += U) {
        Raw8<IO> xr[U][VPT], zr[U][VPT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t token = token0 + (turn + u) * pl.step;
            const bool live = place < pl.count && token < a.tokens;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = (tid + i * TPR) * 8, left = live ? V - c : 0;
                xr[u][i] = load8((const IO*)x.p + token * x.ld + (int64_t)head * V + c, left, x.vec, c);
                zr[u][i] = load8((const IO*)z.p + token * z.ld + (int64_t)head * V + c, left, z.vec, c);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t token = token0 + (turn + u) * pl.step;
            const bool live = place < pl.count && token < a.tokens;
            F2 v[VPT][4], part = both(0.f);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                pairs<IO, 8>(xr[u][i], v[i]);
#pragma unroll
                for (int k = 0; k < 4; ++k) part = fma2(v[i][k], v[i][k], part);
            }
            float sum[1] = {both_halves(part)};
            sum_row<TPR>(sum, red, (int)turn + u);
            const F2 rstd = both(rsqrtf(fmaf(sum[0], over, a.eps)));
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = (tid + i * TPR) * 8;
                F2 zf[4], wf[4];
                pairs<IO, 8>(zr[u][i], zf), pairs<IO, 8>(wr[i], wf);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[i][k] = mul2(mul2(mul2(v[i][k], rstd), wf[k]), gate2<SILU>(zf[k]));
                store_pairs(y + (token * a.H + head) * V + c, v[i], live ? V - c : 0, vec_y);
            }
        }
    }
}

// partial: a row of V sums for each place, or (one weight for all heads, rows of up to a warp) for each block.
template <typename IO, int TPR, int VPT, bool SILU>
__global__ void __launch_bounds__(block_of(TPR), backward_blocks(TPR, VPT))
gated_norm_backward_kernel(GatedNormArgs a, Places pl, const IO* __restrict__ dy, RowTensor x, RowTensor z,
                           const IO* __restrict__ w, IO* __restrict__ dx, IO* __restrict__ dz,
                           float* __restrict__ partial, bool vec_w, bool vec) {
    constexpr int NT = block_of(TPR), RPB = NT / TPR;
    __shared__ float red[2][2 * 32];
    const int tid = threadIdx.x % TPR, V = a.V;
    const int64_t place = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    const int head = (int)(place % a.H);
    const int64_t token0 = place / a.H;
    const IO* wp = w + (a.per_head ? (int64_t)head * V : 0);
    Raw8<IO> wr[VPT], xr[VPT], zr[VPT], gr[VPT];
    F2 dw[VPT][4];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        wr[i] = load8(wp + (tid + i * TPR) * 8, V - (tid + i * TPR) * 8, vec_w, (tid + i * TPR) * 8);
#pragma unroll
        for (int k = 0; k < 4; ++k) dw[i][k] = both(0.f);
    }
    const float over = 1.f / (float)V;
    const auto load = [&](int64_t turn) {
        const int64_t token = token0 + turn * pl.step;
        const bool live = place < pl.count && token < a.tokens;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * TPR) * 8, left = live ? V - c : 0;
            xr[i] = load8((const IO*)x.p + token * x.ld + (int64_t)head * V + c, left, x.vec, c);
            zr[i] = load8((const IO*)z.p + token * z.ld + (int64_t)head * V + c, left, z.vec, c);
            gr[i] = load8(dy + (token * a.H + head) * V + c, left, vec, c);
        }
    };
    load(0);
    for (int64_t turn = 0; turn < pl.turns; ++turn) {
        const int64_t token = token0 + turn * pl.step;
        const bool live = place < pl.count && token < a.tokens;
        F2 xf[VPT][4], gw[VPT][4], f[VPT][4], slope[VPT][4], p0 = both(0.f), p1 = both(0.f);
        Raw8<IO> now[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            F2 zf[4], wf[4];
            now[i] = gr[i];
            pairs<IO, 8>(xr[i], xf[i]), pairs<IO, 8>(zr[i], zf), pairs<IO, 8>(gr[i], gw[i]), pairs<IO, 8>(wr[i], wf);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                gate_and_slope2<SILU>(zf[k], f[i][k], slope[i][k]);
                gw[i][k] = mul2(gw[i][k], wf[k]);
                p0 = fma2(xf[i][k], xf[i][k], p0);
                p1 = fma2(mul2(gw[i][k], f[i][k]), xf[i][k], p1);
            }
        }
        if (turn + 1 < pl.turns) load(turn + 1);             // on their way while this row is worked on
        float sq[1] = {both_halves(p0)}, dot[1] = {both_halves(p1)};
        sum_row<TPR>(sq, red[0], (int)turn);
        sum_row<TPR>(dot, red[1], (int)turn);
        const float rs = live ? rsqrtf(fmaf(sq[0], over, a.eps)) : 0.f;     // with eps = 0 a row that is not there has none
        const F2 rstd = both(rs), back = both(-dot[0] * over * rs * rs);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * TPR) * 8, left = live ? V - c : 0;
            const int64_t at = (token * a.H + head) * V + c;
            F2 g[4], o[4], oz[4];
            pairs<IO, 8>(now[i], g);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const F2 n = mul2(xf[i][k], rstd);
                o[k] = mul2(rstd, fma2(xf[i][k], back, mul2(gw[i][k], f[i][k])));
                oz[k] = mul2(mul2(gw[i][k], n), slope[i][k]);
                dw[i][k] = fma2(mul2(g[k], n), f[i][k], dw[i][k]);          // a row that is not there adds zero
            }
            store_pairs(dx + at, o, left, vec);
            store_pairs(dz + at, oz, left, vec);
        }
    }
    if (TPR <= 32 && !a.per_head) {                          // the block's places, one after another
        __shared__ float sums[TPR <= 32 ? RPB : 1][TPR <= 32 ? TPR * VPT * 8 : 1];
        float* mine = sums[threadIdx.x / TPR];
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 v = unpack2(dw[i][k]);
                mine[(tid + i * TPR) * 8 + 2 * k] = v.x, mine[(tid + i * TPR) * 8 + 2 * k + 1] = v.y;
            }
        __syncthreads();
        for (int c = threadIdx.x; c < V; c += NT) {
            float sum = 0.f;
#pragma unroll
            for (int p = 0; p < RPB; ++p) sum += sums[p][c];
            partial[(int64_t)blockIdx.x * V + c] = sum;
        }
    } else if (place < pl.count) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 q = unpack2(dw[i][k]);
                v[2 * k] = q.x, v[2 * k + 1] = q.y;
            }
            store_cut(partial + place * V, v, (tid + i * TPR) * 8, V, (V & 3) == 0);
        }
    }
}

Shape shape_of(int V) {
    const int v = (V + 7) / 8;
    for (int tpr = 4; tpr <= 256; tpr *= 2)
        if (v <= tpr) return {tpr, 1};
    return {v <= 512 ? 256 : 512, 2};
}

Places places_of(const GatedNormArgs& a, Shape h, int blocks) {
    const int64_t rpb = block_of(h.tpr) / h.tpr, most = (int64_t)kSms * blocks * rpb;
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
    GDR_SHAPE(4, 1) GDR_SHAPE(8, 1) GDR_SHAPE(16, 1) GDR_SHAPE(32, 1) GDR_SHAPE(64, 1) GDR_SHAPE(128, 1) GDR_SHAPE(256, 1)
    GDR_SHAPE(256, 2) GDR_SHAPE(512, 2)
#undef GDR_SHAPE
    return cudaErrorInvalidValue;
}

// Rows of a warp at most, one weight for all heads: one for each block.
bool rows_by_block(const GatedNormArgs& a, Shape h) { return h.tpr <= 32 && !a.per_head; }

// Whether the heads' rows of all these tensors start on 16-byte boundaries.
bool on_16(std::initializer_list<const void*> ps, int64_t head_bytes) {
    bool vec = head_bytes % 16 == 0;
    for (const void* p : ps) vec = vec && reinterpret_cast<uintptr_t>(p) % 16 == 0;
    return vec;
}

}  // namespace

cudaError_t gated_norm_forward(const GatedNormArgs& a, RowTensor x, RowTensor z, const void* w, void* y, cudaStream_t s) {
    const Shape h = shape_of(a.V);
    const Places p = places_of(a, h, forward_blocks(h.tpr, h.vpt));
    return with_types(a, h, [&](auto io, auto tpr, auto vpt, auto silu) {
        using IO = decltype(io);
        constexpr int T = decltype(tpr)::value, NT = block_of(T);
        const int64_t bytes = (int64_t)a.V * sizeof(IO);
        x.vec = x.vec && bytes % 16 == 0, z.vec = z.vec && bytes % 16 == 0;
        gated_norm_forward_kernel<IO, T, decltype(vpt)::value, decltype(silu)::value>
            <<<(unsigned)((p.count + NT / T - 1) / (NT / T)), NT, 0, s>>>(a, p, x, z, (const IO*)w, (IO*)y, on_16({w}, bytes),
                                                                        on_16({y}, bytes));
        return cudaGetLastError();
    });
}

int64_t gated_norm_partial_rows(const GatedNormArgs& a) {
    const Shape h = shape_of(a.V);
    const int64_t places = places_of(a, h, backward_blocks(h.tpr, h.vpt)).count, rpb = block_of(h.tpr) / h.tpr;
    return rows_by_block(a, h) ? (places + rpb - 1) / rpb : places;
}

cudaError_t gated_norm_backward(const GatedNormArgs& a, const void* dy, RowTensor x, RowTensor z, const void* w, void* dx,
                                void* dz, float* dw, float* partial, cudaStream_t s) {
    const Shape h = shape_of(a.V);
    const Places p = places_of(a, h, backward_blocks(h.tpr, h.vpt));
    const cudaError_t e = with_types(a, h, [&](auto io, auto tpr, auto vpt, auto silu) {
        using IO = decltype(io);
        constexpr int T = decltype(tpr)::value, NT = block_of(T);
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
    const int64_t rows = rows_by_block(a, h) ? gated_norm_partial_rows(a) : p.count * a.V / cols;
    return column_sum(partial, rows, cols, cols, dw, 0, nullptr, s);
}

}  // namespace layer
}  // namespace gdr
