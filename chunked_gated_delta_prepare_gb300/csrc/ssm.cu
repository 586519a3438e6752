// The selective state space scan over prompts and for single tokens (ssm.cuh has the formulas).
//
// Bound: an exponential for every token, channel and state, 32 a clock on an SM, and 4 fp32 operations beside it (the
// exponent's and the input's products, the recurrence, the output's sum), which at 128 a clock cost the same.  A thread
// keeps 4 channels x 4 states in registers: 16 independent recurrences hide each other's latency, and only 3 shuffles a
// token join a channel's output.  The inputs of 16 tokens come through shared memory in fp32: softplus, its product
// with x, and the widening happen once a value and not once a state.
//
// Few sequences and channels leave most of the GPU idle, so a long sequence is cut into segments: a first kernel scans
// every segment but the last from a zero state and keeps what it leaves and the sum of its Delta (its decay is
// exp(A sum Delta)); the second starts each segment from its predecessors' states, joined in order, and does the rest.
// That is twice the work, so a batch that fills the GPU without it is scanned whole.
#include <algorithm>

#include "ssm.cuh"

namespace gdr {
namespace layer {
namespace {

constexpr int kTile = 16;          // tokens staged in shared memory
constexpr int kDC = 4;             // channels of a thread
constexpr int kMinSegment = 64;

template <int LN> constexpr int width_of() { return kSsmThreads / LN * kDC; }

// LOCAL: what each segment with a successor leaves from a zero state, into ends [segment][D][N], and its sum of Delta,
// into sums [segment][D].  Else: the scan.
template <typename IO, int LN, bool LOCAL>
__global__ void __launch_bounds__(kSsmThreads)
ssm_scan_kernel(Ssm a, float* __restrict__ ends, float* __restrict__ sums, IO* __restrict__ y,
                float* __restrict__ h_final) {
    constexpr int W = width_of<LN>(), P = kDC / 2;
    __shared__ float4 s_delta[kTile * W / 4], s_u[kTile * W / 4];      // Delta (then y), Delta x
    __shared__ float2 s_b[kTile * 4 * LN], s_c[LOCAL ? 1 : kTile * 4 * LN];
    const TileAt at = find_tile(a.q, blockIdx.x, a.seg);
    if (at.seq < 0) return;
    const bool last = (at.tile + 1) * a.seg >= at.len;
    if (LOCAL && last) return;
    const Channels ch = block_channels(a, W);
    const int q = threadIdx.x % LN, n = 4 * q, own = threadIdx.x / LN * kDC, c = ch.c0 + own;
    const int64_t state = (int64_t)a.D * a.N;

    F2 A2[4][P], h[4][P], sum[P];
    load_decay<kDC>(a, c, ch.end, n, A2);
    load_states<kDC>(LOCAL || !a.h0 ? nullptr : a.h0 + at.seq * state, a, c, ch.end, n, h);
    if (!LOCAL)
        for (int64_t s = (int64_t)blockIdx.x - at.tile; s < (int64_t)blockIdx.x; ++s) {
            F2 e[4][P];
            load_states<kDC>(ends + s * state, a, c, ch.end, n, e);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float* p = sums + s * a.D + c + 2 * i;
                const F2 t = pack2(c + 2 * i < ch.end ? p[0] : 0.f, c + 2 * i + 1 < ch.end ? p[1] : 0.f);
#pragma unroll
                for (int j = 0; j < 4; ++j) h[j][i] = fma2(exp2_2(mul2(A2[j][i], t)), h[j][i], e[j][i]);
            }
        }
#pragma unroll
    for (int i = 0; i < P; ++i) sum[i] = 0;

    const int64_t t0 = at.tile * a.seg, t1 = min(t0 + a.seg, at.len);
    for (int64_t t = t0; t < t1; t += kTile) {
        const int live = (int)min((int64_t)kTile, t1 - t);
        const int64_t row = at.start + t;
        for (int i = threadIdx.x; i < kTile * W / 8; i += kSsmThreads) {
            const int k = i / (W / 8), col = i % (W / 8) * 8, cc = ch.c0 + col;
            const int left = k < live ? ch.end - cc : 0;
            float d[8], u[8];
            widen(load_row8<IO>(a.dt, row + k, cc, left), d);
            widen(load_row8<IO>(a.x, row + k, cc, left), u);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                d[j] = j < left ? step_size(a, d[j], cc + j) : 0.f;      // Delta = 0: the state stays as it is
                u[j] = j < left ? u[j] * d[j] : 0.f;
            }
            float4* pd = s_delta + (k * W + col) / 4;
            float4* pu = s_u + (k * W + col) / 4;
            pd[0] = make_float4(d[0], d[1], d[2], d[3]), pd[1] = make_float4(d[4], d[5], d[6], d[7]);
            pu[0] = make_float4(u[0], u[1], u[2], u[3]), pu[1] = make_float4(u[4], u[5], u[6], u[7]);
        }
        load_bc<IO, LN>(a, a.B, ch.group, row, live, kTile, s_b);
        if (!LOCAL) load_bc<IO, LN>(a, a.C, ch.group, row, live, kTile, s_c);
        __syncthreads();
#pragma unroll 2
        for (int k = 0; k < live; ++k) {
            F2 d[P], u[P], b[4], o[P];
            const F2* pd = reinterpret_cast<const F2*>(s_delta) + (k * W + own) / 2;
            const F2* pu = reinterpret_cast<const F2*>(s_u) + (k * W + own) / 2;
            const F2* pb = reinterpret_cast<const F2*>(s_b) + k * 4 * LN + n;
#pragma unroll
            for (int i = 0; i < P; ++i) d[i] = pd[i], u[i] = pu[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = pb[j];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < P; ++i) h[j][i] = fma2(exp2_2(mul2(A2[j][i], d[i])), h[j][i], mul2(u[i], b[j]));
            if (LOCAL) {
#pragma unroll
                for (int i = 0; i < P; ++i) sum[i] = add2(sum[i], d[i]);
            } else {
                const F2* pc = reinterpret_cast<const F2*>(s_c) + k * 4 * LN + n;
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    o[i] = mul2(h[0][i], pc[0]);
#pragma unroll
                    for (int j = 1; j < 4; ++j) o[i] = fma2(h[j][i], pc[j], o[i]);
                }
                const float2 lo = unpack2(o[0]), hi = unpack2(o[1]);
                float v[4] = {lo.x, lo.y, hi.x, hi.y};
                lanes_sum4<LN>(v, q);          // every lane of the channel has read its Delta by now
                float* out = reinterpret_cast<float*>(s_delta) + k * W + own;
                if (LN == 2) *reinterpret_cast<float2*>(out + 2 * q) = make_float2(v[0], v[1]);
                else if (q < 4) out[keep4(q)] = v[0];
            }
        }
        __syncthreads();
        if (!LOCAL) {
            for (int i = threadIdx.x; i < live * W / 8; i += kSsmThreads) {
                const int k = i / (W / 8), col = i % (W / 8) * 8, cc = ch.c0 + col, left = ch.end - cc;
                if (left <= 0) continue;
                const float4* py = s_delta + (k * W + col) / 4;
                const float4 y0 = py[0], y1 = py[1];
                float o[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w}, v[8];
                if (a.Dk) {
                    widen(load_row8<IO>(a.x, row + k, cc, left), v);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < left) o[j] = fmaf(a.Dk[cc + j], v[j], o[j]);
                }
                if (a.z.p) {
                    widen(load_row8<IO>(a.z, row + k, cc, left), v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] *= v[j] * sigmoid(v[j]);
                }
                store_n(y + (row + k) * a.D + cc, o, left, a.vec && (cc & 7) == 0);
            }
            __syncthreads();
        }
    }
    if (LOCAL) {
        store_states<kDC>(ends + blockIdx.x * state, a, c, ch.end, n, h);
        if (q == 0)
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float2 f = unpack2(sum[i]);
                float* p = sums + (int64_t)blockIdx.x * a.D + c + 2 * i;
                if (c + 2 * i < ch.end) p[0] = f.x;
                if (c + 2 * i + 1 < ch.end) p[1] = f.y;
            }
    } else if (last && h_final) {
        store_states<kDC>(h_final + at.seq * state, a, c, ch.end, n, h);
    }
}

// One token of a row: LN lanes a channel, 4 states each, the state read and written once.
template <typename IO, int LN>
__global__ void __launch_bounds__(256)
ssm_step_kernel(Ssm a, int64_t pool, const int* __restrict__ slots, float* __restrict__ h, IO* __restrict__ y) {
    const int q = threadIdx.x % LN, n = 4 * q, c = blockIdx.y * (256 / LN) + threadIdx.x / LN;
    const int64_t row = blockIdx.x, slot = slots ? slots[row] : row;
    if (slot < 0 || slot >= pool) {
        if (q == 0 && c < a.D) y[row * a.D + c] = from_f<IO>(0.f);
        return;
    }
    const bool in = c < a.D;              // lanes past the last channel stay for the shuffles
    float* hp = h + (slot * a.D + c) * a.N + n;
    const float* Ap = a.A + (int64_t)c * a.N + n;
    const bool whole = in && n + 4 <= a.N && (reinterpret_cast<uintptr_t>(hp) & 15) == 0;
    float s[4], A[4];
    if (whole) {
        const float4 v = *reinterpret_cast<const float4*>(hp);
        s[0] = v.x, s[1] = v.y, s[2] = v.z, s[3] = v.w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = in && n + j < a.N ? hp[j] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) A[j] = in && n + j < a.N ? Ap[j] * kLog2e : 0.f;
    float x = 0.f, d = 0.f, o = 0.f;
    if (in) {
        x = to_f(reinterpret_cast<const IO*>(a.x.p)[row * a.x.ld + c]);
        d = step_size(a, to_f(reinterpret_cast<const IO*>(a.dt.p)[row * a.dt.ld + c]), c);
    }
    const int g = in ? c / a.per : 0;
    const IO* Bp = reinterpret_cast<const IO*>(a.B.p) + row * a.B.ld + g * a.N + n;
    const IO* Cp = reinterpret_cast<const IO*>(a.C.p) + row * a.C.ld + g * a.N + n;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (n + j >= a.N) continue;
        s[j] = fmaf(ex2(A[j] * d), s[j], x * d * to_f(Bp[j]));
        o = fmaf(s[j], to_f(Cp[j]), o);
    }
#pragma unroll
    for (int k = 1; k < LN; k *= 2) o += __shfl_xor_sync(0xffffffffu, o, k);
    if (whole) *reinterpret_cast<float4*>(hp) = make_float4(s[0], s[1], s[2], s[3]);
    else
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (in && n + j < a.N) hp[j] = s[j];
    if (q == 0 && in) {
        if (a.Dk) o = fmaf(a.Dk[c], x, o);
        if (a.z.p) {
            const float z = to_f(reinterpret_cast<const IO*>(a.z.p)[row * a.z.ld + c]);
            o *= z * sigmoid(z);
        }
        y[row * a.D + c] = from_f<IO>(o);
    }
}

int blocks_of_channels(const SsmArgs& a, int width) { return a.G * ((a.D / a.G + width - 1) / width); }

// Tokens of a segment.  A batch whose blocks fill the GPU (4 an SM) is scanned whole; anything else is cut into as many
// segments as give kSms * 8 blocks.
int segment_of(const SsmArgs& a) {
    const int64_t width = kSsmThreads / ssm_lanes(a.N) * kDC, blocks = blocks_of_channels(a, (int)width);
    const int64_t longest = a.cu ? a.total : a.T;
    int64_t seg = longest;
    if (a.cu || a.n * blocks < kSms * 4) seg = std::min(longest, a.total * blocks / (kSms * 8) + 1);
    seg = std::max<int64_t>(seg, kMinSegment);
    return (int)((seg + kTile - 1) / kTile * kTile);
}

}  // namespace

size_t ssm_forward_workspace(const SsmArgs& a) {
    const int seg = segment_of(a);
    if (seg >= (a.cu ? a.total : a.T)) return 0;
    const Seqs q{a.cu, a.total, a.T, (int)a.n};
    return (size_t)tile_count(q, seg) * (size_t)a.D * (size_t)(a.N + 1) * 4;
}

cudaError_t ssm_forward(const SsmArgs& a, const SsmTensors& t, void* y, float* h_final, float* workspace,
                        cudaStream_t s) {
    Ssm k = ssm_of(a, t);
    k.seg = segment_of(a);
    k.vec = (int64_t)a.D * (a.io == GDR_F32 ? 4 : 2) % 16 == 0 && reinterpret_cast<uintptr_t>(y) % 16 == 0;
    const int64_t segments = tile_count(k.q, k.seg);
    const bool split = ssm_forward_workspace(a) > 0;
    float *ends = workspace, *sums = split ? workspace + segments * a.D * a.N : nullptr;
    return ssm_types(a.io, a.N, [&](auto io, auto lanes) {
        using IO = decltype(io);
        constexpr int LN = decltype(lanes)::value;
        const dim3 grid((unsigned)segments, (unsigned)blocks_of_channels(a, width_of<LN>()));
        if (split) {
            ssm_scan_kernel<IO, LN, true><<<grid, kSsmThreads, 0, s>>>(k, ends, sums, nullptr, nullptr);
            if (cudaError_t e = cudaGetLastError()) return e;
        }
        ssm_scan_kernel<IO, LN, false><<<grid, kSsmThreads, 0, s>>>(k, ends, sums, (IO*)y, h_final);
        return cudaGetLastError();
    });
}

cudaError_t ssm_step(const SsmArgs& a, const SsmTensors& t, int64_t pool, const int* slots, float* h, void* y,
                     cudaStream_t s) {
    const Ssm k = ssm_of(a, t);
    return ssm_types(a.io, a.N, [&](auto io, auto lanes) {
        using IO = decltype(io);
        constexpr int LN = decltype(lanes)::value, per = 256 / LN;
        ssm_step_kernel<IO, LN><<<dim3((unsigned)a.n, (unsigned)((a.D + per - 1) / per)), 256, 0, s>>>(k, pool, slots, h,
                                                                                                      (IO*)y);
        return cudaGetLastError();
    });
}

}  // namespace layer
}  // namespace gdr
