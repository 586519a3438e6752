// The layer norm of a row with the residual's addition, and its gradient.
//
//   s = x + residual, m = mean s, rstd = 1 / sqrt(mean (s - m)^2 + eps), y = (s - m) rstd w + b   (fp32, rounded once)
//   xh = (s - m) rstd,  ds = rstd (w dy - mean(w dy) - xh mean(w dy xh)) + dr,  dw = sum dy xh,  db = sum dy
//
// Bound: memory.  A row is read once and stays in registers between its two sums (the mean first, then the squares around
// it: one pass over squares would lose a row whose mean is far from zero) and the output.  With many rows they arrive whole
// by bulk copies, several rows ahead of the threads that work on them.
#include "blackwell.cuh"
#include "gdr_internal.h"
#include "norm.cuh"

namespace gdr {
namespace layer {
namespace {

// ---------------------------------------------------------------- rows through shared memory
//
// A block an SM: its threads make up places of TPR threads, each working on rows of its own with one ring of stages for
// their inputs, so that the barriers of one row hold up no other.  The rows' copies are in flight whatever the threads wait
// for.  768 threads where a row takes at most 256 of them: 80 registers a thread.

constexpr int kMaxStages = 4, kRingBytes = 200 * 1024;
constexpr int ring_block(int tpr) { return tpr <= 256 ? 768 : tpr; }

__device__ __forceinline__ void bulk_load(void* to, const void* from, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(bw::smem_u32(to)),
                 "l"(from), "r"(bytes), "r"(bw::smem_u32(bar))
                 : "memory");
}

// Sums over a place's TPR threads; red: [warps of the block][NV], not used again before another barrier of the place.
template <int TPR, int NV> __device__ __forceinline__ void place_sum(float (&v)[NV], float (*red)[NV]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if (TPR == 32) return;
    constexpr int W = TPR / 32;
    const int warp = threadIdx.x / 32, place = threadIdx.x / TPR, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < NV; ++i) red[warp][i] = v[i];
    bw::named_bar_sync(place + 1, TPR);        // 0 is the block's; at most 12 places
    if (W <= 8) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            v[i] = red[place * W][i];
#pragma unroll
            for (int w = 1; w < W; ++w) v[i] += red[place * W + w][i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float u = lane < W ? red[place * W + lane][i] : 0.f;
#pragma unroll
            for (int o = W / 2; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
            v[i] = __shfl_sync(0xffffffffu, u, 0);
        }
    }
}

// The rows of a place and its ring: T tensors, `stages` rows of each ahead.  A row is copied from the 16-byte boundary at or
// before its start; what a tensor has after its last such boundary is not copied.
template <typename IO, int T> struct Ring {
    const IO* base[T];            // nullptr: not there
    int64_t ld[T];                // elements
    int64_t rows;
    int D, stages;
    uint32_t pitch;               // bytes of a row in shared memory
    unsigned char* smem;          // the place's: [stages][T][pitch]
    uint64_t* full;               // [stages]

    __device__ __forceinline__ const IO* at(int stage, int t) const {
        return reinterpret_cast<const IO*>(smem + (stage * T + t) * pitch);
    }
    // Elements of row `row` that are copied, from the boundary on.
    __device__ __forceinline__ int copied(int64_t row) const {
        constexpr int per = 16 / (int)sizeof(IO);
        const int shift = (int)(row * D % per), n = (shift + D + per - 1) / per * per;
        return row + 1 < rows ? n : (shift + D) / per * per;      // only contiguous rows have a shift
    }
    __device__ __forceinline__ void issue(int64_t row, int stage, bool cut) const {
        if (row >= rows) return;
        const uint32_t bytes = (cut ? copied(row) : D) * (uint32_t)sizeof(IO);
        uint32_t all = 0;
#pragma unroll
        for (int t = 0; t < T; ++t) all += base[t] ? bytes : 0;
        bw::mbar_arrive_expect_tx(full + stage, all);
#pragma unroll
        for (int t = 0; t < T; ++t)
            if (base[t])
                bulk_load(smem + (stage * T + t) * pitch,
                          base[t] + row * ld[t] - (cut ? row * D % (16 / (int)sizeof(IO)) : 0), bytes, full + stage);
    }
};

// The thread's vector of 8 columns from column c = 8 i - shift on; zeros outside the row.
template <typename IO, bool CUT>
__device__ __forceinline__ Raw8<IO> ring_vector(const IO* row, int i, int c, int D, const IO* global, int copied) {
    Raw8<IO> r;
    if (CUT ? c >= D : c + 8 > D) {
        if (!CUT && c < D) {                   // fp32 rows of 4 columns more than a multiple of 8
#pragma unroll
            for (int j = 0; j < 8; ++j) r.e[j] = c + j < D ? row[8 * i + j] : from_f<IO>(0.f);
            return r;
        }
        return load8((const IO*)nullptr, 0, false);
    }
    if (CUT && 8 * i + 8 > copied) return load_cut(global, c, D, false);
#pragma unroll
    for (int k = 0; k < (int)sizeof(r) / 16; ++k)
        reinterpret_cast<uint4*>(&r)[k] = reinterpret_cast<const uint4*>(row + 8 * i)[k];
    if (CUT) mask_cut(r, c, D);
    return r;
}

template <typename IO, int TPR, int VPT, bool CUT>
__global__ void __launch_bounds__(ring_block(TPR), 1)
layernorm_ring_kernel(NormArgs a, RowTensor x, RowTensor res, const IO* __restrict__ w, const IO* __restrict__ b,
                      IO* __restrict__ y, IO* __restrict__ r, int stages, uint32_t pitch, bool vec_w, unsigned* err) {
    constexpr int NT = ring_block(TPR), P = NT / TPR;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float red[2][2][NT / 32][1];
    __shared__ uint64_t full[P][kMaxStages];
    const int tid = threadIdx.x % TPR, place = threadIdx.x / TPR, D = a.D;
    if (threadIdx.x == 0) {
        for (int i = 0; i < P * kMaxStages; ++i) bw::mbar_init(&full[0][0] + i, 1);
        bw::fence_mbar_init();
    }
    __syncthreads();
    const int64_t step = (int64_t)gridDim.x * P, first = (int64_t)blockIdx.x * P + place;
    const Ring<IO, 2> ring{{(const IO*)x.p, (const IO*)res.p}, {x.ld, res.ld}, a.rows, D, stages, pitch,
                           smem + (size_t)place * stages * 2 * pitch, full[place]};
    if (tid == 0)
        for (int k = 0; k < stages; ++k) ring.issue(first + k * step, k, CUT);
    const int shift = CUT ? first_shift<IO>(first, D) : 0;
    Raw8<IO> wr[VPT], br[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (tid + i * TPR) * 8 - shift;
        wr[i] = load_cut(w, c, D, vec_w && shift == 0);
        br[i] = b ? load_cut(b, c, D, vec_w && shift == 0) : load8((const IO*)nullptr, 0, false);
    }
    int stage = 0, phase = 0, turn = 0;
    for (int64_t row = first; row < a.rows; row += step, ++turn) {
        bw::mbar_wait(full[place] + stage, phase, err, kDeviceErrTimeout);
        const int copied = CUT ? ring.copied(row) : 0;
        float v[VPT][8], sum[1] = {0.f}, var[1] = {0.f};
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int n = tid + i * TPR, c = n * 8 - shift;
            widen(ring_vector<IO, CUT>(ring.at(stage, 0), n, c, D, (const IO*)x.p + row * D, copied), v[i]);
            if (res.p) {
                float t[8];
                widen(ring_vector<IO, CUT>(ring.at(stage, 1), n, c, D, (const IO*)res.p + row * D, copied), t);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += t[j];
            }
            if (r) store_cut(r + row * D, v[i], c, D, true);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[0] += v[i][j];
        }
        place_sum<TPR, 1>(sum, red[turn & 1][0]);
        if (tid == 0) ring.issue(row + stages * step, stage, CUT);          // every thread has read the stage
        if (++stage == stages) stage = 0, phase ^= 1;
        const float mean = sum[0] / (float)D;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * TPR) * 8 - shift;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] -= mean;
            if (c < 0 || c + 8 > D)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j < 0 || c + j >= D) v[i][j] = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) var[0] = fmaf(v[i][j], v[i][j], var[0]);
        }
        place_sum<TPR, 1>(var, red[turn & 1][1]);
        const float rstd = rsqrtf(var[0] / (float)D + a.eps);
        if (!y) continue;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * TPR) * 8 - shift;
            float wf[8], bf[8];
            widen(wr[i], wf), widen(br[i], bf);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = fmaf(v[i][j] * rstd, wf[j], bf[j]);
            store_cut(y + row * D, v[i], c, D, true);
        }
    }
}

// One vector a thread, whose sums of dw and db stay in registers; a block leaves one row of partial sums [2 D].
template <typename IO, int TPR, bool CUT>
__global__ void __launch_bounds__(ring_block(TPR), 1)
layernorm_backward_ring_kernel(NormArgs a, const IO* __restrict__ dy, const IO* __restrict__ r, const IO* __restrict__ w,
                               const IO* __restrict__ dr, IO* __restrict__ dx, float* __restrict__ partial, int stages,
                               uint32_t pitch, bool vec_w, unsigned* err) {
    constexpr int NT = ring_block(TPR), P = NT / TPR;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float red[2][2][NT / 32][2];
    __shared__ uint64_t full[P][kMaxStages];
    const int tid = threadIdx.x % TPR, place = threadIdx.x / TPR, D = a.D;
    if (threadIdx.x == 0) {
        for (int i = 0; i < P * kMaxStages; ++i) bw::mbar_init(&full[0][0] + i, 1);
        bw::fence_mbar_init();
    }
    __syncthreads();
    const int64_t step = (int64_t)gridDim.x * P, first = (int64_t)blockIdx.x * P + place;
    const Ring<IO, 3> ring{{dy, r, dr}, {D, D, D}, a.rows, D, stages, pitch, smem + (size_t)place * stages * 3 * pitch,
                           full[place]};
    if (tid == 0)
        for (int k = 0; k < stages; ++k) ring.issue(first + k * step, k, CUT);
    const int shift = CUT ? first_shift<IO>(first, D) : 0, c = tid * 8 - shift;
    const Raw8<IO> wr = load_cut(w, c, D, vec_w && shift == 0);
    float dw[8], db[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[j] = db[j] = 0.f;
    int stage = 0, phase = 0, turn = 0;
    for (int64_t row = first; row < a.rows; row += step, ++turn) {
        bw::mbar_wait(full[place] + stage, phase, err, kDeviceErrTimeout);
        const int copied = CUT ? ring.copied(row) : 0;
        float g[8], s[8], wf[8], o[8], one[2] = {0.f, 0.f}, two[2] = {0.f, 0.f};
        widen(ring_vector<IO, CUT>(ring.at(stage, 0), tid, c, D, dy + row * D, copied), g);
        widen(ring_vector<IO, CUT>(ring.at(stage, 1), tid, c, D, r + row * D, copied), s);
        const Raw8<IO> er = dr ? ring_vector<IO, CUT>(ring.at(stage, 2), tid, c, D, dr + row * D, copied)
                               : load8((const IO*)nullptr, 0, false);
        widen(wr, wf);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            one[0] += s[j];
            one[1] = fmaf(wf[j], g[j], one[1]);
        }
        place_sum<TPR, 2>(one, red[turn & 1][0]);
        if (tid == 0) ring.issue(row + stages * step, stage, CUT);          // every thread has read the stage
        if (++stage == stages) stage = 0, phase ^= 1;
        const float mean = one[0] / (float)D, flat = one[1] / (float)D;
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] -= mean;
        if (c < 0 || c + 8 > D)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j < 0 || c + j >= D) s[j] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            two[0] = fmaf(s[j], s[j], two[0]);
            two[1] = fmaf(wf[j] * g[j], s[j], two[1]);
        }
        place_sum<TPR, 2>(two, red[turn & 1][1]);
        const float rstd = rsqrtf(two[0] / (float)D + a.eps), back = two[1] / (float)D * rstd * rstd;
        widen(er, o);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            o[j] = fmaf(rstd, fmaf(-s[j], back, fmaf(wf[j], g[j], -flat)), o[j]);
            dw[j] = fmaf(g[j], s[j] * rstd, dw[j]);
            db[j] += g[j];
        }
        store_cut(dx + row * D, o, c, D, true);
    }
    // the places' sums, one after another
    __syncthreads();
    float* sums = reinterpret_cast<float*>(smem);            // [2 D], every row has been read
    for (int i = threadIdx.x; i < 2 * D; i += NT) sums[i] = 0.f;
    __syncthreads();
    for (int p = 0; p < P; ++p) {
        if (place == p)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j >= 0 && c + j < D) sums[c + j] += dw[j], sums[D + c + j] += db[j];
        __syncthreads();
    }
    for (int i = threadIdx.x; i < 2 * D; i += NT) partial[(int64_t)blockIdx.x * 2 * D + i] = sums[i];
}

// ---------------------------------------------------------------- rows straight into registers

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

// How rows go through the ring: threads of a row (0: they do not), stages, bytes of a row in shared memory.
struct RingPlan {
    int tpr, stages;
    uint32_t pitch;
    int places() const { return ring_block(tpr) / tpr; }
    int bytes(int tensors) const { return places() * stages * tensors * (int)pitch; }
};
// At least three rows for each place of the GPU: below that nothing is ahead.  vpt: vectors a thread.
RingPlan ring_plan(const NormArgs& a, int tensors, int vpt) {
    RingPlan p{0, 0, 0};
    const int e = a.io == GDR_F32 ? 4 : 2, v = vectors_of(a);
    if (a.D * e < 256) return p;              // copies of a few lines each take longer than loads
    p.tpr = 32;
    while (p.tpr < 1024 && p.tpr * vpt < v) p.tpr *= 2;
    if (p.tpr * vpt < v || a.rows < 3 * p.places() * kSms) return RingPlan{0, 0, 0};
    p.pitch = (uint32_t)((a.D * e + 15 + 16 + 15) / 16 * 16);
    p.stages = std::min<int>(kMaxStages, kRingBytes / (p.places() * tensors * (int)p.pitch));
    if (p.stages < 2) p.tpr = 0;
    return p;
}
// Whether every row starts on a 16-byte boundary (1), or all tensors are contiguous from one on (2).
int ring_rows(const NormArgs& a, std::initializer_list<RowTensor> in, std::initializer_list<const void*> contiguous) {
    const int64_t row = (int64_t)a.D * (a.io == GDR_F32 ? 4 : 2);
    bool whole = row % 16 == 0, cut = true;
    for (const RowTensor& t : in) {
        if (!t.p) continue;
        whole = whole && t.vec;
        cut = cut && t.ld == a.D && reinterpret_cast<uintptr_t>(t.p) % 16 == 0;
    }
    for (const void* p : contiguous) {
        const bool on = reinterpret_cast<uintptr_t>(p) % 16 == 0;
        whole = whole && on, cut = cut && on;
    }
    return whole ? 1 : cut ? 2 : 0;
}
template <typename F> cudaError_t ring_threads(int tpr, F f) {
#define GDR_TPR(T) \
    if (tpr == T) return f(std::integral_constant<int, T>());
    GDR_TPR(32) GDR_TPR(64) GDR_TPR(128) GDR_TPR(256) GDR_TPR(512) GDR_TPR(1024)
#undef GDR_TPR
    return cudaErrorInvalidValue;
}
template <typename F> cudaError_t io_type(int io, F f) {
    if (io == GDR_F32) return f(float());
    if (io == GDR_BF16) return f(__nv_bfloat16());
    return f(__half());
}

}  // namespace

cudaError_t layernorm_forward(const NormArgs& a, RowTensor x, RowTensor res, const void* w, const void* b, void* y,
                              void* r, cudaStream_t s) {
    const int vpt = a.io == GDR_F32 ? 1 : 2, rows = ring_rows(a, {x, res}, {y, r});
    const RingPlan plan = ring_plan(a, 2, vpt);
    if (rows && plan.tpr) {
        unsigned* err = nullptr;
        if (cudaError_t e = device_error_ptr(&err)) return e;
        return ring_threads(plan.tpr, [&](auto tpr) {
            return io_type(a.io, [&](auto io) {
                using IO = decltype(io);
                constexpr int T = decltype(tpr)::value, V = sizeof(IO) == 4 ? 1 : 2;
                const auto go = [&](auto kernel) {
                    const int bytes = plan.bytes(2);
                    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes))
                        return e;
                    kernel<<<kSms, ring_block(T), bytes, s>>>(a, x, res, (const IO*)w, (const IO*)b, (IO*)y, (IO*)r,
                                                             plan.stages, plan.pitch, on_16({w, b}, 16), err);
                    return cudaGetLastError();
                };
                return rows == 1 ? go(layernorm_ring_kernel<IO, T, V, false>) : go(layernorm_ring_kernel<IO, T, V, true>);
            });
        });
    }
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

int64_t layernorm_partial_rows(const NormArgs& a) {      // of either way: which it is depends on the pointers
    const Shape h = shape_of(a.D);
    return std::max<int64_t>(ring_plan(a, 3, 1).tpr ? kSms : 0, grid_of(a, h) * (h.tpr < 128 ? 128 / h.tpr : 1));
}

cudaError_t layernorm_backward(const NormArgs& a, const void* dy, const void* r, const void* w, const void* dr, void* dx,
                               float* dw, float* db, float* partial, cudaStream_t s) {
    const RowTensor none{nullptr, 0, false};
    const int rows = ring_rows(a, {none}, {dy, r, dr, dx});
    const RingPlan plan = ring_plan(a, 3, 1);
    if (rows && plan.tpr) {
        unsigned* err = nullptr;
        if (cudaError_t e = device_error_ptr(&err)) return e;
        const cudaError_t e = ring_threads(plan.tpr, [&](auto tpr) {
            return io_type(a.io, [&](auto io) {
                using IO = decltype(io);
                constexpr int T = decltype(tpr)::value;
                const auto go = [&](auto kernel) {
                    const int bytes = std::max(plan.bytes(3), 8 * a.D);
                    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes))
                        return e;
                    kernel<<<kSms, ring_block(T), bytes, s>>>(a, (const IO*)dy, (const IO*)r, (const IO*)w, (const IO*)dr,
                                                             (IO*)dx, partial, plan.stages, plan.pitch, on_16({w}, 16), err);
                    return cudaGetLastError();
                };
                return rows == 1 ? go(layernorm_backward_ring_kernel<IO, T, false>)
                                 : go(layernorm_backward_ring_kernel<IO, T, true>);
            });
        });
        if (e != cudaSuccess) return e;
        return column_sum(partial, kSms, 2 * (int64_t)a.D, a.D, dw, a.D, db, s);
    }
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
    return column_sum(partial, grid_of(a, h) * (h.tpr < 128 ? 128 / h.tpr : 1), 2 * (int64_t)a.D, a.D, dw, a.D, db, s);
}

}  // namespace layer
}  // namespace gdr
