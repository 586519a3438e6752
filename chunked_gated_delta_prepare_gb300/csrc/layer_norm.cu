// The layer norm of a row with the residual's addition, and its gradient.
//
//   s = x + residual, m = mean s, rstd = 1 / sqrt(mean (s - m)^2 + eps), y = (s - m) rstd w + b   (fp32, rounded once)
//   xh = (s - m) rstd,  ds = rstd (w dy - mean(w dy) - xh mean(w dy xh)) + dr,  dw = sum dy xh,  db = sum dy
//
// Bound: memory.  A row is read once and stays in registers between its two sums (the mean first, then the squares around
// it: one pass over squares would lose a row whose mean is far from zero) and the output.  With many rows they arrive whole
// by bulk copies, several rows ahead of the threads that work on them.
//
// Measured (bf16): 32768 x 4096 with residual in 185 us, 5.8 TB/s, 0.86 of a copy's rate (277 by loads into registers);
// 8192 x 2048 forward 22, gradient 28 and 3 for column_sum; 4451 x 2278 fp32, rows that start between boundaries, 72 in all.
// The gradient has 16 warps an SM (dw and db take 32 registers of a thread's 120) and issues in 0.47 of its slots: each
// instruction less shows.  One barrier a row instead of two, by joining the warps' own means and squares, takes more of them
// and measured slower (16384 x 2048: 62 us against 57).
#include "blackwell.cuh"
#include "gdr_internal.h"
#include "norm.cuh"

namespace gdr {
namespace layer {
namespace {

// ---------------------------------------------------------------- rows through shared memory
//
// A block an SM: its threads make up places of `tpr` threads, each working on rows of its own with one ring of stages for
// their inputs, so that the barriers of one row hold up no other.  The rows' copies are in flight whatever the threads wait
// for.

constexpr int kMaxStages = 4, kRingBytes = 200 * 1024;
constexpr int kForwardWarps = 24, kBackwardWarps = 16;       // of a block: 80 and 128 registers a thread
constexpr int kBackwardVectors = 2;                          // a thread

__device__ __forceinline__ void bulk_load(void* to, const void* from, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(bw::smem_u32(to)), "l"(from), "r"(bytes), "r"(bw::smem_u32(bar))
                 : "memory");
}

constexpr int ring_places(int warps, int most) { return (warps <= most ? most : 32) / warps; }
// A place's rows are kSms places apart times a block's: where rows are cut at the boundaries, their shift, and with it the
// columns of the weights and sums in a thread's registers, repeats after at most 8 rows.
static_assert(kSms % 8 == 0, "every row of a place has the shift of its first");

// Sums over a place's WARPS warps; red: [NV][places][WARPS, a multiple of 4], zero where there is no warp, not used again
// before another barrier of the place.
template <int WARPS, int P> constexpr int kRedSlots = P * ((WARPS + 3) / 4 * 4);
template <int WARPS, int NV, int SLOTS> __device__ __forceinline__ void place_sum(float (&v)[NV], float (*red)[SLOTS]) {
    static_assert(NV == 1 || NV == 2, "one sum a lane, or one a half of the warp");
    const int lane = threadIdx.x & 31;
    float sum = v[0];
    if (NV == 2) {                                          // the halves take a sum each
        const bool second = lane & 16;
        sum = second ? v[NV - 1] : v[0];
        sum += __shfl_xor_sync(0xffffffffu, second ? v[0] : v[NV - 1], 16);
    }
#pragma unroll
    for (int o = NV == 2 ? 8 : 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (WARPS == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = NV == 1 ? sum : __shfl_sync(0xffffffffu, sum, 16 * i);
        return;
    }
    constexpr int slots = (WARPS + 3) / 4 * 4;
    const int warp = threadIdx.x / 32, place = warp / WARPS;
    if (lane % (32 / NV) == 0) red[lane / (32 / NV)][place * slots + warp % WARPS] = sum;
    bw::named_bar_sync(place + 1, WARPS * 32);              // 0 is the block's; at most 12 places of two warps and more
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const float4* q = reinterpret_cast<const float4*>(red[i] + place * slots);
        v[i] = 0.f;
#pragma unroll
        for (int w = 0; w < slots / 4; ++w) {
            const float4 f = q[w];
            v[i] += (f.x + f.y) + (f.z + f.w);
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

// The thread's vector of 8 columns from column c = 8 i - shift on; zeros outside the row.  Rows that are not cut have zeros
// behind them (clear_ends), so that no thread asks where they end.
template <typename IO, bool CUT>
__device__ __forceinline__ Raw8<IO> ring_vector(const IO* row, int i, int c, int D, const IO* global, int copied) {
    Raw8<IO> r;
    if (CUT && c >= D) return load8((const IO*)nullptr, 0, false);
    if (CUT && 8 * i + 8 > copied) return load_cut(global, c, D, false);
    const IO* from = row + (CUT ? 8 * i : min(c, D));
#pragma unroll
    for (int k = 0; k < (int)sizeof(r) / 16; ++k) reinterpret_cast<uint4*>(&r)[k] = reinterpret_cast<const uint4*>(from)[k];
    if (CUT) mask_cut(r, c, D);
    return r;
}
// The 32 bytes behind each of n rows that are not cut.
__device__ __forceinline__ void clear_ends(unsigned char* smem, int n, uint32_t pitch, uint32_t bytes, int threads) {
    for (int i = threadIdx.x; i < 2 * n; i += threads)
        *reinterpret_cast<uint4*>(smem + (i >> 1) * pitch + bytes + (i & 1) * 16) = make_uint4(0, 0, 0, 0);
}

// v + less in the columns of the row, zero outside.
template <typename IO, bool CUT> __device__ __forceinline__ void shift_columns(F2 (&v)[4], float less, int c, int D) {
    // not cut: whole halves of a vector, or (16 bits) whole vectors, are there or not
    const float lo = CUT || c < D ? less : 0.f, hi = CUT ? less : sizeof(IO) == 2 ? lo : c + 4 < D ? less : 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = add2(v[k], both(k < 2 ? lo : hi));
    if (CUT && (c < 0 || c + 8 > D))
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = unpack2(v[k]);
            const int at = c + 2 * k;
            v[k] = pack2(at >= 0 && at < D ? f.x : 0.f, at + 1 >= 0 && at + 1 < D ? f.y : 0.f);
        }
}
__device__ __forceinline__ float both_halves(F2 v) {
    const float2 f = unpack2(v);
    return f.x + f.y;
}
template <typename IO, bool CUT> __device__ __forceinline__ void store_pairs(IO* row, const F2 (&v)[4], int c, int D) {
    float x[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 f = unpack2(v[k]);
        x[2 * k] = f.x, x[2 * k + 1] = f.y;
    }
    if (CUT) return store_cut(row, x, c, D, true);
    Raw8<IO> r;
#pragma unroll
    for (int i = 0; i < 8; i += 2) from_f2(r.e + i, x[i], x[i + 1]);
#pragma unroll
    for (int k = 0; k < (int)sizeof(r) / 16; ++k)
        if (c + 4 * k < D) reinterpret_cast<uint4*>(row + c)[k] = reinterpret_cast<const uint4*>(&r)[k];
}

template <typename IO, int WARPS, int VPT, bool CUT>
__global__ void __launch_bounds__(ring_places(WARPS, kForwardWarps) * WARPS * 32, 1)
layernorm_ring_kernel(NormArgs a, RowTensor x, RowTensor res, const IO* __restrict__ w, const IO* __restrict__ b,
                      IO* __restrict__ y, IO* __restrict__ r, int stages, uint32_t pitch, bool vec_w,
                      unsigned* err) {
    constexpr int P = ring_places(WARPS, kForwardWarps), tpr = WARPS * 32, NT = P * tpr;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ __align__(16) float red[2][2][1][kRedSlots<WARPS, P>];
    __shared__ uint64_t full[P][kMaxStages];
    const int tid = threadIdx.x % tpr, place = threadIdx.x / tpr, D = a.D;
    for (int i = threadIdx.x; i < 4 * kRedSlots<WARPS, P>; i += NT) (&red[0][0][0][0])[i] = 0.f;
    if (!CUT) clear_ends(smem, P * stages * 2, pitch, D * (uint32_t)sizeof(IO), NT);
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
        const int c = (tid + i * tpr) * 8 - shift;
        wr[i] = load_cut(w, c, D, vec_w && shift == 0);
        br[i] = b ? load_cut(b, c, D, vec_w && shift == 0) : load8((const IO*)nullptr, 0, false);
    }
    const float over = 1.f / (float)D;
    int stage = 0, phase = 0, turn = 0;
    for (int64_t row = first; row < a.rows; row += step, ++turn) {
        bw::mbar_wait(full[place] + stage, phase, err, kDeviceErrTimeout);
        const int copied = CUT ? ring.copied(row) : 0;
        F2 v[VPT][4], part = both(0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int n = tid + i * tpr, c = n * 8 - shift;
            pairs<IO, 8>(ring_vector<IO, CUT>(ring.at(stage, 0), n, c, D, (const IO*)x.p + row * D, copied), v[i]);
            if (res.p) {
                F2 t[4];
                pairs<IO, 8>(ring_vector<IO, CUT>(ring.at(stage, 1), n, c, D, (const IO*)res.p + row * D, copied), t);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[i][k] = add2(v[i][k], t[k]);
            }
            if (r) store_pairs<IO, CUT>(r + row * D, v[i], c, D);
#pragma unroll
            for (int k = 0; k < 4; ++k) part = add2(part, v[i][k]);
        }
        float sum[1] = {both_halves(part)};
        place_sum<WARPS, 1>(sum, red[turn & 1][0]);
        if (tid == 0) ring.issue(row + stages * step, stage, CUT);          // every thread has read the stage
        if (++stage == stages) stage = 0, phase ^= 1;
        part = both(0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            shift_columns<IO, CUT>(v[i], -sum[0] * over, (tid + i * tpr) * 8 - shift, D);
#pragma unroll
            for (int k = 0; k < 4; ++k) part = fma2(v[i][k], v[i][k], part);
        }
        float var[1] = {both_halves(part)};
        place_sum<WARPS, 1>(var, red[turn & 1][1]);
        const F2 rstd = both(rsqrtf(fmaf(var[0], over, a.eps)));
        if (!y) continue;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            F2 wf[4], bf[4];
            pairs<IO, 8>(wr[i], wf), pairs<IO, 8>(br[i], bf);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[i][k] = fma2(mul2(v[i][k], rstd), wf[k], bf[k]);
            store_pairs<IO, CUT>(y + row * D, v[i], (tid + i * tpr) * 8 - shift, D);
        }
    }
}

// The sums of dw and db stay in registers; a block leaves one row of partial sums [2 D].
template <typename IO, int WARPS, int VPT, bool CUT>
__global__ void __launch_bounds__(ring_places(WARPS, kBackwardWarps) * WARPS * 32, 1)
layernorm_backward_ring_kernel(NormArgs a, const IO* __restrict__ dy, const IO* __restrict__ r, const IO* __restrict__ w,
                               const IO* __restrict__ dr, IO* __restrict__ dx, float* __restrict__ partial, int stages,
                               uint32_t pitch, bool vec_w, unsigned* err) {
    constexpr int P = ring_places(WARPS, kBackwardWarps), tpr = WARPS * 32, NT = P * tpr;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ __align__(16) float red[2][2][2][kRedSlots<WARPS, P>];
    __shared__ uint64_t full[P][kMaxStages];
    const int tid = threadIdx.x % tpr, place = threadIdx.x / tpr, D = a.D;
    for (int i = threadIdx.x; i < 8 * kRedSlots<WARPS, P>; i += NT) (&red[0][0][0][0])[i] = 0.f;
    if (!CUT) clear_ends(smem, P * stages * 3, pitch, D * (uint32_t)sizeof(IO), NT);
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
    const int shift = CUT ? first_shift<IO>(first, D) : 0;
    F2 wf[VPT][4], dw[VPT][4], db[VPT][4];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        pairs<IO, 8>(load_cut(w, (tid + i * tpr) * 8 - shift, D, vec_w && shift == 0), wf[i]);
#pragma unroll
        for (int k = 0; k < 4; ++k) dw[i][k] = db[i][k] = both(0.f);
    }
    const float over = 1.f / (float)D;
    int stage = 0, phase = 0, turn = 0;
    for (int64_t row = first; row < a.rows; row += step, ++turn) {
        bw::mbar_wait(full[place] + stage, phase, err, kDeviceErrTimeout);
        const int copied = CUT ? ring.copied(row) : 0;
        F2 g[VPT][4], s[VPT][4], p0 = both(0.f), p1 = both(0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int n = tid + i * tpr, c = n * 8 - shift;
            pairs<IO, 8>(ring_vector<IO, CUT>(ring.at(stage, 0), n, c, D, dy + row * D, copied), g[i]);
            pairs<IO, 8>(ring_vector<IO, CUT>(ring.at(stage, 1), n, c, D, r + row * D, copied), s[i]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                p0 = add2(p0, s[i][k]);
                p1 = fma2(wf[i][k], g[i][k], p1);
            }
        }
        float one[2] = {both_halves(p0), both_halves(p1)};
        place_sum<WARPS, 2>(one, red[turn & 1][0]);
        // every thread is done with the row before: its stage is free
        if (tid == 0 && turn > 0) ring.issue(row + (stages - 1) * step, stage == 0 ? stages - 1 : stage - 1, CUT);
        const F2 flat = both(-one[1] * over);
        p0 = p1 = both(0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            shift_columns<IO, CUT>(s[i], -one[0] * over, (tid + i * tpr) * 8 - shift, D);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                p0 = fma2(s[i][k], s[i][k], p0);
                p1 = fma2(mul2(wf[i][k], g[i][k]), s[i][k], p1);
            }
        }
        float two[2] = {both_halves(p0), both_halves(p1)};
        place_sum<WARPS, 2>(two, red[turn & 1][1]);
        const float rs = rsqrtf(fmaf(two[0], over, a.eps));
        const F2 rstd = both(rs), back = both(-two[1] * over * rs * rs);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int n = tid + i * tpr, c = n * 8 - shift;
            F2 o[4];
            pairs<IO, 8>(dr ? ring_vector<IO, CUT>(ring.at(stage, 2), n, c, D, dr + row * D, copied)
                            : load8((const IO*)nullptr, 0, false), o);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                o[k] = fma2(rstd, fma2(s[i][k], back, fma2(wf[i][k], g[i][k], flat)), o[k]);
                dw[i][k] = fma2(g[i][k], mul2(s[i][k], rstd), dw[i][k]);
                db[i][k] = add2(db[i][k], g[i][k]);
            }
            store_pairs<IO, CUT>(dx + row * D, o, c, D);
        }
        if (++stage == stages) stage = 0, phase ^= 1;
    }
    // the places' sums, one after another
    __syncthreads();
    float* sums = reinterpret_cast<float*>(smem);            // [2 D], every row has been read
    for (int i = threadIdx.x; i < 2 * D; i += NT) sums[i] = 0.f;
    __syncthreads();
    for (int p = 0; p < P; ++p) {
        if (place == p)
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 fw = unpack2(dw[i][k]), fb = unpack2(db[i][k]);
                    const int at = (tid + i * tpr) * 8 - shift + 2 * k;
                    if (at >= 0 && at < D) sums[at] += fw.x, sums[D + at] += fb.x;
                    if (at + 1 >= 0 && at + 1 < D) sums[at + 1] += fw.y, sums[D + at + 1] += fb.y;
                }
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

// How rows go through the ring: warps of a row (0: they do not), stages, bytes of a row in shared memory.
struct RingPlan {
    int warps = 0, stages = 0;
    uint32_t pitch = 0;
    int bytes(int tensors, int most) const { return ring_places(warps, most) * stages * tensors * (int)pitch; }
};
// At least three rows for each place of the GPU: below that nothing is ahead.  vpt: vectors a thread; most: a block's warps.
RingPlan ring_plan(const NormArgs& a, int tensors, int vpt, int most) {
    RingPlan p;
    const int e = a.io == GDR_F32 ? 4 : 2, need = (vectors_of(a) + 32 * vpt - 1) / (32 * vpt);
    if (a.D * e < 256) return p;              // copies of a few lines each take longer than loads
    for (int w : {1, 2, 3, 4, 6, 8, 12, 16, 32})
        if (w >= need && !p.warps) p.warps = w;
    if (!p.warps) return p;
    const int places = ring_places(p.warps, most);
    p.pitch = (uint32_t)((a.D * e + 15 + 16 + 15) / 16 * 16);
    p.stages = std::min<int>(kMaxStages, kRingBytes / (places * tensors * (int)p.pitch));
    if (p.stages < 2 || a.rows < 3 * places * kSms) return RingPlan();
    return p;
}
template <typename F> cudaError_t ring_warps(int warps, F f) {
#define GDR_WARPS(W) \
    if (warps == W) return f(std::integral_constant<int, W>());
    GDR_WARPS(1) GDR_WARPS(2) GDR_WARPS(3) GDR_WARPS(4) GDR_WARPS(6) GDR_WARPS(8) GDR_WARPS(12) GDR_WARPS(16) GDR_WARPS(32)
#undef GDR_WARPS
    return cudaErrorInvalidValue;
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
template <typename F> cudaError_t io_type(int io, F f) {
    if (io == GDR_F32) return f(float());
    if (io == GDR_BF16) return f(__nv_bfloat16());
    return f(__half());
}

}  // namespace

cudaError_t layernorm_forward(const NormArgs& a, RowTensor x, RowTensor res, const void* w, const void* b, void* y,
                              void* r, cudaStream_t s) {
    const int vpt = a.io == GDR_F32 ? 1 : 2, rows = ring_rows(a, {x, res}, {y, r});
    const RingPlan plan = ring_plan(a, 2, vpt, kForwardWarps);
    if (rows && plan.warps) {
        unsigned* err = nullptr;
        if (cudaError_t e = device_error_ptr(&err)) return e;
        return ring_warps(plan.warps, [&](auto warps) {
            return io_type(a.io, [&](auto io) {
                using IO = decltype(io);
                constexpr int W = decltype(warps)::value, V = sizeof(IO) == 4 ? 1 : 2;
                const auto go = [&](auto kernel) {
                    const int bytes = plan.bytes(2, kForwardWarps);
                    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes))
                        return e;
                    kernel<<<kSms, ring_places(W, kForwardWarps) * W * 32, bytes, s>>>(
                        a, x, res, (const IO*)w, (const IO*)b, (IO*)y, (IO*)r, plan.stages, plan.pitch, on_16({w, b}, 16), err);
                    return cudaGetLastError();
                };
                return rows == 1 ? go(layernorm_ring_kernel<IO, W, V, false>) : go(layernorm_ring_kernel<IO, W, V, true>);
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
    const bool ring = ring_plan(a, 3, kBackwardVectors, kBackwardWarps).warps > 0;
    return std::max<int64_t>(ring ? kSms : 0, grid_of(a, h) * (h.tpr < 128 ? 128 / h.tpr : 1));
}

cudaError_t layernorm_backward(const NormArgs& a, const void* dy, const void* r, const void* w, const void* dr, void* dx,
                               float* dw, float* db, float* partial, cudaStream_t s) {
    const RowTensor none{nullptr, 0, false};
    const int rows = ring_rows(a, {none}, {dy, r, dr, dx});
    const RingPlan plan = ring_plan(a, 3, kBackwardVectors, kBackwardWarps);
    if (rows && plan.warps) {
        unsigned* err = nullptr;
        if (cudaError_t e = device_error_ptr(&err)) return e;
        const cudaError_t e = ring_warps(plan.warps, [&](auto warps) {
            return io_type(a.io, [&](auto io) {
                using IO = decltype(io);
                constexpr int W = decltype(warps)::value;
                const auto go = [&](auto kernel) {
                    const int bytes = std::max(plan.bytes(3, kBackwardWarps), 8 * a.D);
                    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes))
                        return e;
                    kernel<<<kSms, ring_places(W, kBackwardWarps) * W * 32, bytes, s>>>(
                        a, (const IO*)dy, (const IO*)r, (const IO*)w, (const IO*)dr, (IO*)dx, partial, plan.stages, plan.pitch,
                        on_16({w}, 16), err);
                    return cudaGetLastError();
                };
                return rows == 1 ? go(layernorm_backward_ring_kernel<IO, W, kBackwardVectors, false>)
                                 : go(layernorm_backward_ring_kernel<IO, W, kBackwardVectors, true>);
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
