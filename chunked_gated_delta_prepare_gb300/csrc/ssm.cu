// The selective state space scan over prompts and for single tokens (ssm.cuh has the formulas).
//
// Bound: an exponential for every token, channel and state, 32 a clock on an SM, and 4 fp32 operations beside it (the
// exponent's and the input's products, the recurrence, the output's sum), which at 128 a clock cost the same; next come
// issue slots and the bytes that shared memory returns to registers.  A thread keeps 4 channels x 8 states: 32
// independent recurrences hide each other's latency, what it reads of a token (Delta and Delta x of its channels, B and C
// of its states, 96 bytes) serves all of them, and 2 shuffles join its channels' outputs.  (4 x 4 took 96 bytes for half
// as many and measured 1.3 times the time.)  Products go two states at a time.  The inputs of a few tokens come through
// shared memory in fp32: softplus, its product with x, and the widening happen once a value and not once a state.  The
// next tile's loads are in flight meanwhile.  Measured: 32768 tokens x 4096 channels x 16 states bf16 652 us, 3.3 T
// exponentials/s of the 9.4 T/s that they reach alone.  That is neither pipe's limit: a warp's token is 64 packed fp32
// instructions and 32 exponentials, 128 cycles of each pipe side by side, and takes about 365 to 390 (3449 warp-tokens a
// scheduler).  Some 210 of these issue, half of them staging, moves, loads and shuffles; the rest is latency that 12 warps
// an SM do not hide.
//
// Few sequences and channels leave most of the GPU idle, so a long sequence is cut into segments: a first kernel scans
// every segment but the last from a zero state and keeps what it leaves and the sum of its Delta (its decay is
// exp(A sum Delta)); a small one joins these in order to the state before each segment; the third scans all segments
// from there.  That is twice the work, so a batch that fills the GPU without it is scanned whole.  (The same prompt: 468 us
// for the first kernel, 9 for the join.)
#include <algorithm>

#include "ssm.cuh"

namespace gdr {
namespace layer {
namespace {

constexpr int kThreads = 128;
constexpr int kMinSegment = 32;
constexpr int kBlocksPerSm = 3;

// Channels of a thread (with a lane a channel 4 would make the tiles of a block too wide) and of a block.
template <int LN> constexpr int channels_of() { return LN == 1 ? 2 : 4; }
template <int LN> constexpr int width_of() { return kThreads / LN * channels_of<LN>(); }
// Tokens staged in shared memory: 8, and 16 where a block has only 64 channels, so that each thread has a vector of 8
// channels to stage (8192 x 4096 x 64 bf16: 1108 us for the scan with 8, 919 with 16).
template <int LN> constexpr int tile_of() { return LN < 8 ? 8 : 16; }

// Sums over a channel's LN lanes of v[0 .. DC), one for each of DC channels.  Partners halve the channels between them
// while there is more than one: lane q is left with those from kept(q) on in v[0 .. kKept).
template <int LN, int DC> struct ChannelSum {
    static constexpr int kKept = LN >= DC ? 1 : DC / LN;
    static __device__ __forceinline__ int kept(int q) {
        int at = 0;
#pragma unroll
        for (int m = 1, size = DC / 2; m < LN && size > 0; m *= 2, size /= 2) at += q & m ? size : 0;
        return at;
    }
    static __device__ __forceinline__ void sum(float (&v)[DC], int q) {
#pragma unroll
        for (int m = 1, size = DC / 2; m < LN; m *= 2, size /= 2) {
            if (size == 0) {
                v[0] += __shfl_xor_sync(0xffffffffu, v[0], m);
            } else {
                const bool up = q & m;
#pragma unroll
                for (int i = 0; i < DC / 2; ++i) {
                    if (i >= size) break;
                    const float give = up ? v[i] : v[i + size], keep = up ? v[i + size] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, give, m);
                }
            }
        }
    }
};

// LOCAL: what each segment with a successor leaves from a zero state, into ends [segment][D][N], and its sum of Delta,
// into sums [segment][D].  Else: the scan.
template <typename IO, int LN, bool LOCAL>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
ssm_scan_kernel(Ssm a, float* __restrict__ ends, float* __restrict__ sums, IO* __restrict__ y,
                float* __restrict__ h_final) {
    constexpr int DC = channels_of<LN>(), W = width_of<LN>(), V8 = W / 8, NP = 8 * LN, kTile = tile_of<LN>();
    constexpr int U = kTile * V8 <= kThreads ? 1 : kTile * V8 / kThreads;     // 8-channel units of a thread
    constexpr int M = (kTile * NP + kThreads - 1) / kThreads;                 // values of B (and of C) of a thread
    using Sum = ChannelSum<LN, DC>;
    __shared__ float4 s_delta[kTile * W / 4], s_u[kTile * W / 4];             // Delta (then y), Delta x
    __shared__ float4 s_b[kTile * NP / 4], s_c[LOCAL ? 1 : kTile * NP / 4];
    __shared__ float4 s_bias[W / 4], s_D[W / 4];
    const TileAt at = find_tile(a.q, blockIdx.x, a.seg);
    if (at.seq < 0) return;
    const bool last = (at.tile + 1) * a.seg >= at.len;
    if (LOCAL && last) return;
    const Channels ch = block_channels(a, W);
    const int q = threadIdx.x % LN, n = 8 * q, own = threadIdx.x / LN * DC, c = ch.c0 + own;
    const int64_t state = (int64_t)a.D * a.N;
    const int64_t t0 = at.tile * a.seg, t1 = min(t0 + a.seg, at.len);

    // Loads of a tile run one tile ahead, those of z from the tile's start.  Unit i of a thread: 8 channels of a token.
    const int col = threadIdx.x % V8 * 8, cc = ch.c0 + col, tok = threadIdx.x / V8;
    const bool vec8 = cc % (16 / (int)sizeof(IO)) == 0;
    Raw8<IO> dt_r[U], x_r[U], x_now[U], z_r[U];
    IO b_r[M], c_r[M];
    const auto fetch = [&](int64_t t) {
        const int64_t row = at.start + t;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int k = tok + i * (kThreads / V8), left = t + k < t1 && k < kTile ? ch.end - cc : 0;
            dt_r[i] = load8(reinterpret_cast<const IO*>(a.dt.p) + (row + k) * a.dt.ld + cc, left, a.dt.vec && vec8, cc);
            x_r[i] = load8(reinterpret_cast<const IO*>(a.x.p) + (row + k) * a.x.ld + cc, left, a.x.vec && vec8, cc);
        }
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const int k = (threadIdx.x + i * kThreads) / NP, m = (threadIdx.x + i * kThreads) % NP;
            const bool in = k < kTile && t + k < t1 && m < a.N;
            const int at_n = ch.group * a.N + m;
            b_r[i] = in ? reinterpret_cast<const IO*>(a.B.p)[(row + k) * a.B.ld + at_n] : from_f<IO>(0.f);
            if (!LOCAL) c_r[i] = in ? reinterpret_cast<const IO*>(a.C.p)[(row + k) * a.C.ld + at_n] : from_f<IO>(0.f);
        }
    };
    fetch(t0);
    for (int i = threadIdx.x; i < W; i += kThreads) {
        const bool in = ch.c0 + i < ch.end;
        reinterpret_cast<float*>(s_bias)[i] = in && a.bias ? a.bias[ch.c0 + i] : 0.f;
        reinterpret_cast<float*>(s_D)[i] = in && a.Dk ? a.Dk[ch.c0 + i] : 0.f;
    }
    F2 A2[DC][4], h[DC][4];
    float sum[DC];
    load_decay<DC, 8>(a, c, ch.end, n, A2);
#pragma unroll
    for (int i = 0; i < DC; ++i) sum[i] = 0.f;
    const float* from = a.h0 ? a.h0 + at.seq * state : nullptr;
    if (LOCAL) from = nullptr;
    else if (at.tile > 0) from = ends + blockIdx.x * state;        // ssm_join_kernel has put it there
    load_states<DC, 8>(from, a, c, ch.end, n, h);
    __syncthreads();

    for (int64_t t = t0; t < t1; t += kTile) {
        const int live = (int)min((int64_t)kTile, t1 - t);
        const int64_t row = at.start + t;
        {
            F2 d[U][4], u[U][4];               // all units side by side: their chains hide each other's latency
            const F2* bias = reinterpret_cast<const F2*>(s_bias) + col / 2;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                x_now[i] = x_r[i];
                pairs(dt_r[i], d[i]);
                pairs(x_r[i], u[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) d[i][j] = add2(d[i][j], bias[j]);
            }
            if (a.softplus)
#pragma unroll
                for (int i = 0; i < U; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) d[i][j] = softplus2(d[i][j]);
            if (tok < kTile)
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const int at_k = ((tok + i * (kThreads / V8)) * W + col) / 2;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        reinterpret_cast<F2*>(s_delta)[at_k + j] = d[i][j];
                        reinterpret_cast<F2*>(s_u)[at_k + j] = mul2(u[i][j], d[i][j]);
                    }
                }
        }
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const int at_n = threadIdx.x + i * kThreads;
            if (kTile * NP % kThreads != 0 && at_n >= kTile * NP) break;
            reinterpret_cast<float*>(s_b)[at_n] = to_f(b_r[i]);
            if (!LOCAL) reinterpret_cast<float*>(s_c)[at_n] = to_f(c_r[i]);
        }
        __syncthreads();
        if (t + kTile < t1) fetch(t + kTile);
        if (!LOCAL && a.z.p)
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int k = tok + i * (kThreads / V8);
                z_r[i] = load8(reinterpret_cast<const IO*>(a.z.p) + (row + k) * a.z.ld + cc, k < live ? ch.end - cc : 0,
                               a.z.vec && vec8, cc);
            }
#pragma unroll 1
        for (int k = 0; k < live; ++k) {
            float d[DC], u[DC], v[DC];
            F2 b[4];
            const float* pd = reinterpret_cast<const float*>(s_delta) + k * W + own;
            const float* pu = reinterpret_cast<const float*>(s_u) + k * W + own;
            const F2* pb = reinterpret_cast<const F2*>(s_b) + (k * NP + n) / 2;
#pragma unroll
            for (int i = 0; i < DC; ++i) d[i] = pd[i], u[i] = pu[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = pb[j];
#pragma unroll
            for (int i = 0; i < DC; ++i) {
                const F2 dd = pack2(d[i], d[i]), uu = pack2(u[i], u[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) h[i][j] = fma2(decay2(A2[i][j], dd), h[i][j], mul2(uu, b[j]));
                if (LOCAL) sum[i] += d[i];
            }
            if (!LOCAL) {
                const F2* pc = reinterpret_cast<const F2*>(s_c) + (k * NP + n) / 2;
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = pc[j];
#pragma unroll
                for (int i = 0; i < DC; ++i) {
                    F2 o = mul2(h[i][0], b[0]);
#pragma unroll
                    for (int j = 1; j < 4; ++j) o = fma2(h[i][j], b[j], o);
                    const float2 f = unpack2(o);
                    v[i] = f.x + f.y;
                }
                Sum::sum(v, q);                // every lane of the channel has read its Delta by now
                if (q < DC)
#pragma unroll
                    for (int i = 0; i < Sum::kKept; ++i)
                        reinterpret_cast<float*>(s_delta)[k * W + own + Sum::kept(q) + i] = v[i];
            }
        }
        __syncthreads();
        if (!LOCAL && tok < kTile) {           // a thread reads the units that it alone writes next
            F2 v[U][4], x[4];
            const F2* D = reinterpret_cast<const F2*>(s_D) + col / 2;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                pairs(x_now[i], x);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[i][j] = reinterpret_cast<const F2*>(s_delta)[((tok + i * (kThreads / V8)) * W + col) / 2 + j];
                if (a.Dk)
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[i][j] = fma2(D[j], x[j], v[i][j]);
            }
            if (a.z.p)
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    pairs(z_r[i], x);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[i][j] = mul2(v[i][j], mul2(x[j], sigmoid2(x[j])));
                }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int k = tok + i * (kThreads / V8);
                float o[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) o[2 * j] = unpack2(v[i][j]).x, o[2 * j + 1] = unpack2(v[i][j]).y;
                store_n(y + (row + k) * a.D + cc, o, k < live ? ch.end - cc : 0, a.vec && vec8);
            }
        }
    }
    if (LOCAL) {
        store_states<DC, 8>(ends + blockIdx.x * state, a, c, ch.end, n, h);
        if (q == 0)
#pragma unroll
            for (int i = 0; i < DC; ++i)
                if (c + i < ch.end) sums[(int64_t)blockIdx.x * a.D + c + i] = sum[i];
    } else if (last && h_final) {
        store_states<DC, 8>(h_final + at.seq * state, a, c, ch.end, n, h);
    }
}

// One thread a channel and state, the segments of blockIdx.y's sequence in order, 8 loads in flight.  blockIdx.z = 0:
// ends, forward; 1: dends, backward (see ssm_join).
__global__ void __launch_bounds__(128)
ssm_join_kernel(Ssm a, float* __restrict__ ends, float* __restrict__ dends, const float* __restrict__ sums,
                const float* __restrict__ dh_final, bool first_whole) {
    constexpr int B = 8;
    const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x, state = (int64_t)a.D * a.N;
    if (i >= state) return;
    const int d = (int)(i / a.N);
    const int seq = a.first_seq + blockIdx.y;
    int64_t start, len;
    seq_range(a.q, seq, &start, &len);
    const int64_t first = first_tile(a.q, seq, a.seg), count = (len + a.seg - 1) / a.seg;
    if (count < 2) return;
    const bool back = blockIdx.z == 1;
    const float A2 = a.A[i] * kLog2e;
    float* v = back ? dends : ends;
    const float* from = back ? dh_final : a.h0;
    float h = from ? from[seq * state + i] : 0.f;
    // step s: the value at segment `at(s)` becomes h, then h goes through that segment; the last needs no step
    const auto at = [&](int64_t s) { return first + (back ? count - 1 - s : s); };
    for (int64_t s0 = 0; s0 + 1 < count; s0 += B) {
        float e[B], t[B];
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const bool in = s0 + k + 1 < count;
            e[k] = in ? v[at(s0 + k) * state + i] : 0.f;
            t[k] = in ? sums[at(s0 + k) * a.D + d] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < B; ++k) {
            if (s0 + k + 1 >= count) break;
            v[at(s0 + k) * state + i] = h;
            h = first_whole && !back && s0 + k == 0 ? e[k] : fmaf(ex2(A2 * t[k]), h, e[k]);
        }
    }
    v[at(count - 1) * state + i] = h;
}

// One token of a row: LN lanes a channel, 8 states each, the state read and written once.  What is left beside the
// state's bytes (softplus, the gate, addresses) is a channel's, so 8 states a thread halve it against 4.  Bound: memory's
// latency, one load of everything a thread: 64 x 4096 x 16 bf16 9.7 us, 3.7 TB/s (10.8 with 4 states a thread; 14.3 with 4
// rows a thread that share A, which leave a quarter of the threads).  That latency counts three times: 4096 blocks at 56
// registers are three waves of 9 an SM, and a block has nothing under way beside its one round of loads.
template <typename IO, int LN>
__global__ void __launch_bounds__(kThreads)
ssm_step_kernel(Ssm a, int64_t pool, const int* __restrict__ slots, float* __restrict__ h, IO* __restrict__ y) {
    const int q = threadIdx.x % LN, n = 8 * q, c = blockIdx.y * (kThreads / LN) + threadIdx.x / LN;
    const int64_t row = blockIdx.x, slot = slots ? slots[row] : row;
    const bool in = c < a.D;              // lanes past the last channel stay for the shuffles
    if (slot < 0 || slot >= pool) {
        if (q == 0 && in) y[row * a.D + c] = from_f<IO>(0.f);
        return;
    }
    float* hp = h + slot * a.D * a.N;
    F2 s[1][4], A2[1][4], b[4], cv[4];
    load_states<1, 8>(hp, a, c, a.D, n, s);
    load_decay<1, 8>(a, c, a.D, n, A2);
    const int g = in ? c / a.per : 0;
    const bool vec = (a.N & 7) == 0;
    pairs(load8(reinterpret_cast<const IO*>(a.B.p) + row * a.B.ld + g * a.N + n, a.N - n, vec && a.B.vec), b);
    pairs(load8(reinterpret_cast<const IO*>(a.C.p) + row * a.C.ld + g * a.N + n, a.N - n, vec && a.C.vec), cv);
    float x = 0.f, d = 0.f, z = 0.f;
    if (in) {
        x = to_f(reinterpret_cast<const IO*>(a.x.p)[row * a.x.ld + c]);
        d = step_size(a, to_f(reinterpret_cast<const IO*>(a.dt.p)[row * a.dt.ld + c]), c);
        if (a.z.p) z = to_f(reinterpret_cast<const IO*>(a.z.p)[row * a.z.ld + c]);
    }
    const F2 dd = both(d), uu = both(x * d);
    F2 sum = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        s[0][j] = fma2(decay2(A2[0][j], dd), s[0][j], mul2(uu, b[j]));
        sum = fma2(s[0][j], cv[j], sum);
    }
    const float2 f = unpack2(sum);
    float o = f.x + f.y;
#pragma unroll
    for (int k = 1; k < LN; k *= 2) o += __shfl_xor_sync(0xffffffffu, o, k);
    store_states<1, 8>(hp, a, c, a.D, n, s);
    if (q == 0 && in) {
        if (a.Dk) o = fmaf(a.Dk[c], x, o);
        if (a.z.p) o *= z * sigmoid(z);
        y[row * a.D + c] = from_f<IO>(o);
    }
}

int width_at(int N) {
    switch (ssm_lanes(N, 8)) {
        case 1: return width_of<1>();
        case 2: return width_of<2>();
        case 4: return width_of<4>();
        default: return width_of<8>();
    }
}

// Tokens of a segment.  A batch whose blocks fill half the GPU is scanned whole; anything else is cut into segments that
// make one wave of blocks (a few blocks more would take a second wave's time).  Packed sequences have up to n segments
// beside those of their tokens; the tokens get at least half the wave.
int segment_of(const SsmArgs& a) {
    const int tile = ssm_lanes(a.N, 8) < 8 ? tile_of<1>() : tile_of<8>();
    const int64_t blocks = ssm_blocks(a, width_at(a.N)), wave = kSms * kBlocksPerSm;
    if (!a.cu && a.n * blocks >= wave / 2) return (int)((a.T + tile - 1) / tile * tile);
    const int64_t all = std::max<int64_t>(wave / blocks, 1);
    const int64_t cuts = a.cu ? std::max<int64_t>(all - a.n, (all + 1) / 2) : std::max<int64_t>(all / a.n, 1);
    const int64_t tokens = a.cu ? a.total : a.T;
    const int64_t seg = std::max<int64_t>((tokens + cuts - 1) / cuts, kMinSegment);
    return (int)((seg + tile - 1) / tile * tile);
}

}  // namespace

cudaError_t ssm_join(const Ssm& a, float* ends, float* dends, const float* sums, const float* dh_final, bool first_whole,
                     cudaStream_t s) {
    const int64_t states = (int64_t)a.D * a.N;
    // sequences are one extent of a grid of at most 65535: more go in several launches
    for (int n0 = 0; n0 < a.q.n; n0 += 65535) {
        Ssm k = a;
        k.first_seq = n0;
        const dim3 grid((unsigned)((states + 127) / 128), (unsigned)std::min(a.q.n - n0, 65535), dends ? 2 : 1);
        ssm_join_kernel<<<grid, 128, 0, s>>>(k, ends, dends, sums, dh_final, first_whole);
        if (cudaError_t e = cudaGetLastError()) return e;
    }
    return cudaSuccess;
}

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
    return ssm_types<8>(a.io, a.N, [&](auto io, auto lanes) {
        using IO = decltype(io);
        constexpr int LN = decltype(lanes)::value;
        const dim3 grid((unsigned)segments, (unsigned)ssm_blocks(a, width_at(a.N)));
        if (split) {
            ssm_scan_kernel<IO, LN, true><<<grid, kThreads, 0, s>>>(k, ends, sums, nullptr, nullptr);
            if (cudaError_t e = cudaGetLastError()) return e;
            if (cudaError_t e = ssm_join(k, ends, nullptr, sums, nullptr, false, s)) return e;
        }
        ssm_scan_kernel<IO, LN, false><<<grid, kThreads, 0, s>>>(k, ends, sums, (IO*)y, h_final);
        return cudaGetLastError();
    });
}

cudaError_t ssm_step(const SsmArgs& a, const SsmTensors& t, int64_t pool, const int* slots, float* h, void* y,
                     cudaStream_t s) {
    const Ssm k = ssm_of(a, t);
    return ssm_types<8>(a.io, a.N, [&](auto io, auto lanes) {
        using IO = decltype(io);
        constexpr int LN = decltype(lanes)::value, per = kThreads / LN;
        ssm_step_kernel<IO, LN>
            <<<dim3((unsigned)a.n, (unsigned)((a.D + per - 1) / per)), kThreads, 0, s>>>(k, pool, slots, h, (IO*)y);
        return cudaGetLastError();
    });
}

}  // namespace layer
}  // namespace gdr
