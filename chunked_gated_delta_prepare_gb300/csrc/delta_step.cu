// The gated delta rule for one token of each row of a batch, the states in a pool and changed in place:
//
//   S~ = D S,  delta = beta (v - S~^T k),  S = S~ + k delta^T,  o = scale S^T q
//
// Bound: memory, each state read once and written once.  The columns of S (the value dimension) do not mix, so a block
// takes 32 of them for one (row, value head): 4 times the blocks of one a head, which fills the GPU at a few heads.
// 8 threads hold a row's 32 columns (16 bytes each), 16 such groups share the K rows; K / 16 16-byte loads a thread are
// in flight at once and the state stays in registers between its load and its store.  With
// S^T q = S~^T q + (k.q) delta both sums over K come from one pass and need one barrier.  Measured: 128 rows of 32 value
// heads, K = V = 128, a gate for each key dimension 94 us, 5.8 TB/s (0.87 of a copy's rate); one row 2.7 us.
#include "layer_common.cuh"
#include "layer_internal.h"

namespace gdr {
namespace layer {
namespace {

constexpr int kThreads = 128, kCols = 32, kLanes = kCols / 4, kGroups = kThreads / kLanes;

template <typename IO, int K, bool PER_K>
__global__ void __launch_bounds__(kThreads)
delta_step_kernel(DeltaStepArgs a, const int* __restrict__ slots, const IO* __restrict__ q, const IO* __restrict__ k,
                  const IO* __restrict__ v, const float* __restrict__ g, const IO* __restrict__ beta,
                  float* __restrict__ h, IO* __restrict__ o) {
    constexpr int R = K / kGroups;
    __shared__ float red[kThreads / 32][kLanes][9];
    const int slices = a.V / kCols;
    const int slice = blockIdx.x % slices, hv = blockIdx.x / slices % a.HV;
    const int64_t b = blockIdx.x / slices / a.HV;
    const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes, warp = threadIdx.x / 32;
    const int c = slice * kCols + lane * 4;
    IO* op = o + (b * a.HV + hv) * a.V + c;
    const int64_t slot = slots ? slots[b] : b;
    if (slot < 0 || slot >= a.pool) {
        if (group == 0)
#pragma unroll
            for (int j = 0; j < 4; ++j) op[j] = from_f<IO>(0.f);
        return;
    }
    float4* hp = reinterpret_cast<float4*>(h + ((slot * a.HV + hv) * K + group) * a.V + c);
    const int64_t step = (int64_t)kGroups * a.V / 4;
    float4 s[R];
#pragma unroll
    for (int i = 0; i < R; ++i) s[i] = hp[i * step];
    const int hk = hv / (a.HV / a.H);
    const IO* qp = q + b * a.q_ld + (int64_t)hk * K + group;
    const IO* kp = k + b * a.k_ld + (int64_t)hk * K + group;
    float kf[R], x[9];                       // S~^T k, S~^T q (4 columns each), k.q
    {
        float qf[R], d[PER_K ? R : 1];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            kf[i] = to_f(kp[i * kGroups]);
            qf[i] = to_f(qp[i * kGroups]);
            if (PER_K) d[i] = expf(g[(b * a.HV + hv) * K + group + i * kGroups]);
        }
        if (!PER_K) d[0] = expf(g[b * a.HV + hv]);
#pragma unroll
        for (int j = 0; j < 9; ++j) x[j] = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float e = d[PER_K ? i : 0];
            s[i].x *= e, s[i].y *= e, s[i].z *= e, s[i].w *= e;
            const float t[4] = {s[i].x, s[i].y, s[i].z, s[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[j] = fmaf(t[j], kf[i], x[j]);
                x[4 + j] = fmaf(t[j], qf[i], x[4 + j]);
            }
            x[8] = fmaf(kf[i], qf[i], x[8]);
        }
    }
    const float bt = to_f(beta[b * a.HV + hv]);
    const IO* vp = v + b * a.v_ld + (int64_t)hv * a.V + c;
    float vf[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) vf[j] = to_f(vp[j]);
#pragma unroll
    for (int j = 0; j < 9; ++j) {
        x[j] += __shfl_xor_sync(0xffffffffu, x[j], 8);
        x[j] += __shfl_xor_sync(0xffffffffu, x[j], 16);
    }
    if (threadIdx.x % 32 < kLanes)
#pragma unroll
        for (int j = 0; j < 9; ++j) red[warp][lane][j] = x[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 9; ++j) {
        x[j] = red[0][lane][j];
#pragma unroll
        for (int i = 1; i < kThreads / 32; ++i) x[j] += red[i][lane][j];
    }
    float delta[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) delta[j] = bt * (vf[j] - x[j]);
#pragma unroll
    for (int i = 0; i < R; ++i)
        hp[i * step] = make_float4(fmaf(kf[i], delta[0], s[i].x), fmaf(kf[i], delta[1], s[i].y),
                                   fmaf(kf[i], delta[2], s[i].z), fmaf(kf[i], delta[3], s[i].w));
    if (group == 0)
#pragma unroll
        for (int j = 0; j < 4; ++j) op[j] = from_f<IO>(a.scale * fmaf(x[8], delta[j], x[4 + j]));
}

}  // namespace

cudaError_t delta_step(const DeltaStepArgs& a, const int* slots, const void* q, const void* k, const void* v,
                       const float* g, const void* beta, float* h, void* o, cudaStream_t s) {
    const unsigned grid = (unsigned)(a.B * a.HV * (a.V / kCols));
    const auto launch = [&](auto io, auto K, auto per_k) {
        using IO = decltype(io);
        delta_step_kernel<IO, decltype(K)::value, decltype(per_k)::value><<<grid, kThreads, 0, s>>>(
            a, slots, (const IO*)q, (const IO*)k, (const IO*)v, g, (const IO*)beta, h, (IO*)o);
        return cudaGetLastError();
    };
    const auto sizes = [&](auto io) {
        const std::integral_constant<int, 64> k64;
        const std::integral_constant<int, 128> k128;
        if (a.K == 64) return a.per_k ? launch(io, k64, std::true_type()) : launch(io, k64, std::false_type());
        return a.per_k ? launch(io, k128, std::true_type()) : launch(io, k128, std::false_type());
    };
    if (a.io == GDR_F32) return sizes(float());
    if (a.io == GDR_BF16) return sizes(__nv_bfloat16());
    return sizes(__half());
}

}  // namespace layer
}  // namespace gdr
