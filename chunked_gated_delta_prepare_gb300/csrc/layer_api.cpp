// The C ABI of the layer operators (include/gdr.h, "the layer around the recurrence"): argument validation,
// workspace planning and dispatch.  Every step of the arithmetic runs in the kernels.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "gdr.h"
#include "layer_internal.h"

using namespace gdr::layer;

namespace {

int64_t element_size(int dtype) { return dtype == GDR_F32 ? 4 : 2; }

bool known_dtype(int dtype) { return dtype == GDR_F32 || dtype == GDR_BF16 || dtype == GDR_F16; }

struct Ptr {
    const void* p;
    int64_t align;
    bool required;
};

gdr_status check(std::initializer_list<Ptr> ptrs) {
    for (const Ptr& q : ptrs)
        if (q.required && !q.p) return GDR_ERR_NULL;
    for (const Ptr& q : ptrs)
        if (reinterpret_cast<uintptr_t>(q.p) % (uintptr_t)q.align) return GDR_ERR_ALIGN;
    return GDR_OK;
}

gdr_status check_workspace(const void* ws, size_t have, size_t need) {
    if (need == 0) return GDR_OK;
    if (!ws || have < need) return GDR_ERR_WORKSPACE;
    return reinterpret_cast<uintptr_t>(ws) % 256 ? GDR_ERR_ALIGN : GDR_OK;
}

RowTensor rows_of(const void* p, int64_t ld, int64_t columns, int64_t e) {
    RowTensor t{p, ld ? ld : columns, false};
    t.vec = reinterpret_cast<uintptr_t>(p) % 16 == 0 && t.ld * e % 16 == 0;
    return t;
}

// Rows of `columns` elements at stride ld (0: contiguous) whose offsets stay far from 64 bits.
bool good_ld(int64_t ld, int64_t columns, int64_t rows) {
    return (ld == 0 || ld >= columns) && (rows <= 0 || ld <= (int64_t{1} << 60) / rows);
}

gdr_status done(cudaError_t e, const char* variant) {
    if (e != cudaSuccess) return GDR_ERR_CUDA;
    gdr::set_last_variant(variant);
    return GDR_OK;
}

// Rows of any tensor, and sequences: the kernels number up to two tiles a token in 31 bits (one for the tokens, one for a
// sequence's end), and round the lengths of segments up in them.
constexpr int64_t kMaxTokens = int64_t{1} << 30;

gdr_status norm_args(const gdr_norm_problem* p, NormArgs* a) {
    if (!p) return GDR_ERR_NULL;
    if (!known_dtype(p->io_dtype)) return GDR_ERR_DTYPE;
    if (p->rows < 0 || p->rows >= kMaxTokens || p->D < 1 || p->D > kNormMaxD) return GDR_ERR_SHAPE;
    if (!good_ld(p->x_ld, p->D, p->rows) || !good_ld(p->res_ld, p->D, p->rows)) return GDR_ERR_SHAPE;
    if (p->group != 0 && p->group != 32 && p->group != 64 && p->group != 128) return GDR_ERR_ARG;
    if (!(p->eps >= 0.f) || std::isinf(p->eps)) return GDR_ERR_ARG;
    *a = NormArgs{p->rows, (int)p->D, p->group, p->eps, p->io_dtype};
    return GDR_OK;
}

// n sequences of T tokens, or packed on `total`: the tokens of the axis, or -1.
int64_t token_axis(int64_t n, int64_t T, int64_t total, bool packed) {
    if (n < 1 || n >= kMaxTokens) return -1;
    if (packed) return total >= 0 && total < kMaxTokens ? total : -1;
    return T >= 1 && T <= (kMaxTokens - 1) / n ? n * T : -1;
}

constexpr int64_t kMaxChannels = int64_t{1} << 20;

gdr_status conv_args(const gdr_conv_problem* p, const int32_t* cu, bool packed, ConvArgs* a) {
    if (!p) return GDR_ERR_NULL;
    if (!known_dtype(p->io_dtype)) return GDR_ERR_DTYPE;
    const int64_t tokens = token_axis(p->n, p->T, p->total, packed);
    if (tokens < 0 || p->D < 1 || p->D > kMaxChannels || !good_ld(p->x_ld, p->D, tokens)) return GDR_ERR_SHAPE;
    if (p->W < kConvMinW || p->W > kConvMaxW) return GDR_ERR_SHAPE;
    if (p->silu != 0 && p->silu != 1) return GDR_ERR_ARG;
    *a = ConvArgs{p->n, p->T, tokens, cu, p->D, p->W, p->io_dtype, p->silu == 1};
    return GDR_OK;
}

gdr_status ssm_args(const gdr_ssm_problem* p, const int32_t* cu, bool packed, SsmArgs* a) {
    if (!p) return GDR_ERR_NULL;
    if (!known_dtype(p->io_dtype)) return GDR_ERR_DTYPE;
    const int64_t tokens = token_axis(p->n, p->T, p->total, packed);
    if (tokens < 0 || p->D < 1 || p->D > kMaxChannels || p->N < 1 || p->N > kSsmMaxN) return GDR_ERR_SHAPE;
    // the blocks of channels of all groups, and those of all channels, are one extent of a grid
    if (p->G < 1 || p->D % p->G || p->G * ((p->D / p->G + kSsmMinWidth - 1) / kSsmMinWidth) > 65535)
        return GDR_ERR_SHAPE;
    for (int64_t ld : {p->x_ld, p->dt_ld, p->z_ld})
        if (!good_ld(ld, p->D, tokens)) return GDR_ERR_SHAPE;
    if (!good_ld(p->b_ld, p->G * p->N, tokens) || !good_ld(p->c_ld, p->G * p->N, tokens)) return GDR_ERR_SHAPE;
    if (p->softplus != 0 && p->softplus != 1) return GDR_ERR_ARG;
    *a = SsmArgs{p->n, p->T, tokens, cu, (int)p->D, (int)p->N, (int)p->G, p->io_dtype, p->softplus == 1};
    return GDR_OK;
}

SsmTensors ssm_tensors(const gdr_ssm_problem* p, const void* x, const void* dt, const float* A, const void* B,
                       const void* C, const float* Dk, const void* z, const float* dt_bias, const float* h0) {
    const int64_t e = element_size(p->io_dtype), bc = p->G * p->N;
    return SsmTensors{rows_of(x, p->x_ld, p->D, e), rows_of(dt, p->dt_ld, p->D, e), rows_of(z, p->z_ld, p->D, e),
                      rows_of(B, p->b_ld, bc, e),   rows_of(C, p->c_ld, bc, e),     A, dt_bias, Dk, h0};
}

}  // namespace

extern "C" {

gdr_status gdr_norm_forward(const gdr_norm_problem* p, const void* x, const void* residual, const void* w, void* y,
                            void* r, void* y8, float* scales, void* stream) {
    NormArgs a;
    if (gdr_status st = norm_args(p, &a)) return st;
    if (p->rows == 0) return GDR_OK;
    const int64_t e = element_size(p->io_dtype);
    if (gdr_status st = check({{x, e, true}, {residual, e, false}, {w, e, true}, {y, e, false}, {r, e, false},
                               {y8, 1, scales != nullptr}, {scales, 4, y8 != nullptr}}))
        return st;
    if (!y && !r && !y8) return GDR_ERR_NULL;
    return done(norm_forward(a, rows_of(x, p->x_ld, p->D, e), rows_of(residual, p->res_ld, p->D, e), w, y, r, y8,
                             scales, (cudaStream_t)stream),
                "norm");
}

size_t gdr_norm_backward_workspace_bytes(const gdr_norm_problem* p) {
    NormArgs a;
    if (norm_args(p, &a)) return 0;
    return (size_t)norm_partial_rows(a) * (size_t)p->D * 4;
}

gdr_status gdr_norm_backward(const gdr_norm_problem* p, const void* dy, const void* r, const void* w, const void* dr,
                             void* dx, float* dw, void* workspace, size_t workspace_bytes, void* stream) {
    NormArgs a;
    if (gdr_status st = norm_args(p, &a)) return st;
    const int64_t e = element_size(p->io_dtype);
    const bool any = p->rows > 0;
    if (gdr_status st =
            check({{dy, e, any}, {r, e, any}, {w, e, true}, {dr, e, false}, {dx, e, any}, {dw, 4, true}}))
        return st;
    if (gdr_status st = check_workspace(workspace, workspace_bytes, gdr_norm_backward_workspace_bytes(p))) return st;
    if (!any)   // the sum of no rows
        return done(cudaMemsetAsync(dw, 0, (size_t)p->D * 4, (cudaStream_t)stream), "norm");
    return done(norm_backward(a, dy, r, w, dr, dx, dw, (float*)workspace, (cudaStream_t)stream), "norm");
}

gdr_status gdr_conv_forward(const gdr_conv_problem* p, const int32_t* cu_seqlens, const void* x, const void* w,
                            const void* b, const void* state, void* y, void* state_out, void* stream) {
    ConvArgs a;
    if (gdr_status st = conv_args(p, cu_seqlens, cu_seqlens != nullptr, &a)) return st;
    const int64_t e = element_size(p->io_dtype);
    const bool any = a.total > 0;
    if (gdr_status st = check({{cu_seqlens, 4, false}, {x, e, any}, {w, e, true}, {b, e, false}, {state, e, false},
                               {y, e, any}, {state_out, e, false}}))
        return st;
    return done(conv_forward(a, rows_of(x, p->x_ld, p->D, e), w, b, state, y, state_out, (cudaStream_t)stream), "conv");
}

size_t gdr_conv_backward_workspace_bytes(const gdr_conv_problem* p, int32_t packed) {
    ConvArgs a;
    const int32_t some = 0;
    if (conv_args(p, packed ? &some : nullptr, packed != 0, &a)) return 0;
    return (size_t)conv_partial_rows(a) * (size_t)(p->D * (p->W + 1)) * 4;
}

gdr_status gdr_conv_backward(const gdr_conv_problem* p, const int32_t* cu_seqlens, const void* x, const void* w,
                             const void* b, const void* state, const void* dy, const void* d_state_out, void* dx,
                             float* dw, float* db, void* d_state, void* workspace, size_t workspace_bytes,
                             void* stream) {
    ConvArgs a;
    if (gdr_status st = conv_args(p, cu_seqlens, cu_seqlens != nullptr, &a)) return st;
    const int64_t e = element_size(p->io_dtype);
    const bool any = a.total > 0;
    if (gdr_status st = check({{cu_seqlens, 4, false}, {x, e, any}, {w, e, true}, {b, e, false}, {state, e, false},
                               {dy, e, any}, {d_state_out, e, false}, {dx, e, any}, {dw, 4, true}, {db, 4, true},
                               {d_state, e, false}}))
        return st;
    const size_t need = gdr_conv_backward_workspace_bytes(p, cu_seqlens != nullptr);
    if (gdr_status st = check_workspace(workspace, workspace_bytes, need)) return st;
    return done(conv_backward(a, rows_of(x, p->x_ld, p->D, e), w, b, state, dy, d_state_out, dx, dw, db, d_state,
                              (float*)workspace, (cudaStream_t)stream),
                "conv");
}

gdr_status gdr_conv_step(const gdr_conv_problem* p, const int32_t* slots, const void* x, const void* w, const void* b,
                         void* state, void* y, void* stream) {
    if (!p) return GDR_ERR_NULL;
    gdr_conv_problem one = *p;
    one.T = 1;
    ConvArgs a;
    if (gdr_status st = conv_args(&one, nullptr, false, &a)) return st;
    if (p->pool < 1 || p->pool >= kMaxTokens || (!slots && p->n > p->pool)) return GDR_ERR_SHAPE;
    const int64_t e = element_size(p->io_dtype);
    if (gdr_status st = check({{slots, 4, false}, {x, e, true}, {w, e, true}, {b, e, false}, {state, e, true},
                               {y, e, true}}))
        return st;
    return done(conv_step(a, p->pool, slots, rows_of(x, p->x_ld, p->D, e), w, b, state, y, (cudaStream_t)stream),
                "conv_step");
}

gdr_status gdr_delta_step(const gdr_step_problem* p, const int32_t* slots, const void* q, const void* k, const void* v,
                          const float* g, const void* beta, float* h, void* o, void* stream) {
    if (!p) return GDR_ERR_NULL;
    if (!known_dtype(p->io_dtype)) return GDR_ERR_DTYPE;
    if (p->gate != GDR_GATE_SCALAR && p->gate != GDR_GATE_PER_K) return GDR_ERR_DTYPE;
    const int64_t HV = p->HV ? p->HV : p->H;
    if (p->B < 1 || p->H < 1 || HV < 1 || HV % p->H || HV > 65535 || p->pool < 1 || p->pool >= kMaxTokens)
        return GDR_ERR_SHAPE;
    if ((p->K != 64 && p->K != 128) || (p->V != 64 && p->V != 128)) return GDR_ERR_SHAPE;
    if (p->B > (kMaxTokens - 1) / (HV * (p->V / 32)) || (!slots && p->B > p->pool)) return GDR_ERR_SHAPE;
    if (!good_ld(p->q_ld, p->H * p->K, p->B) || !good_ld(p->k_ld, p->H * p->K, p->B) ||
        !good_ld(p->v_ld, HV * p->V, p->B))
        return GDR_ERR_SHAPE;
    if (std::isnan(p->scale) || std::isinf(p->scale)) return GDR_ERR_ARG;
    const int64_t e = element_size(p->io_dtype);
    if (gdr_status st = check({{slots, 4, false}, {q, e, true}, {k, e, true}, {v, e, true}, {g, 4, true},
                               {beta, e, true}, {h, 16, true}, {o, e, true}}))
        return st;
    const DeltaStepArgs a{p->B, p->pool, (int)p->H, (int)HV, (int)p->K, (int)p->V,
                          p->q_ld ? p->q_ld : p->H * p->K, p->k_ld ? p->k_ld : p->H * p->K,
                          p->v_ld ? p->v_ld : HV * p->V,
                          p->scale > 0.f ? p->scale : 1.f / std::sqrt((float)p->K), p->io_dtype,
                          p->gate == GDR_GATE_PER_K};
    return done(delta_step(a, slots, q, k, v, g, beta, h, o, (cudaStream_t)stream), "delta_step");
}

size_t gdr_ssm_forward_workspace_bytes(const gdr_ssm_problem* p, int32_t packed) {
    SsmArgs a;
    const int32_t some = 0;
    if (ssm_args(p, packed ? &some : nullptr, packed != 0, &a)) return 0;
    return ssm_forward_workspace(a);
}

gdr_status gdr_ssm_forward(const gdr_ssm_problem* p, const int32_t* cu_seqlens, const void* x, const void* dt,
                           const float* A, const void* B, const void* C, const float* Dk, const void* z,
                           const float* dt_bias, const float* h0, void* y, float* h_final, void* workspace,
                           size_t workspace_bytes, void* stream) {
    SsmArgs a;
    if (gdr_status st = ssm_args(p, cu_seqlens, cu_seqlens != nullptr, &a)) return st;
    const int64_t e = element_size(p->io_dtype);
    const bool any = a.total > 0;
    if (gdr_status st = check({{cu_seqlens, 4, false}, {x, e, any}, {dt, e, any}, {A, 4, true}, {B, e, any}, {C, e, any},
                               {Dk, 4, false}, {z, e, false}, {dt_bias, 4, false}, {h0, 4, false}, {y, e, any},
                               {h_final, 4, false}}))
        return st;
    if (gdr_status st = check_workspace(workspace, workspace_bytes, ssm_forward_workspace(a))) return st;
    return done(ssm_forward(a, ssm_tensors(p, x, dt, A, B, C, Dk, z, dt_bias, h0), y, h_final, (float*)workspace,
                            (cudaStream_t)stream),
                ssm_forward_workspace(a) ? "ssm_segments" : "ssm");
}

size_t gdr_ssm_backward_workspace_bytes(const gdr_ssm_problem* p, int32_t packed) {
    SsmArgs a;
    const int32_t some = 0;
    if (ssm_args(p, packed ? &some : nullptr, packed != 0, &a)) return 0;
    return ssm_backward_workspace(a);
}

gdr_status gdr_ssm_backward(const gdr_ssm_problem* p, const int32_t* cu_seqlens, const void* x, const void* dt,
                            const float* A, const void* B, const void* C, const float* Dk, const void* z,
                            const float* dt_bias, const float* h0, const void* dy, const float* dh_final, void* dx,
                            void* ddt, float* dA, void* dB, void* dC, float* dDk, void* dz, float* ddt_bias, float* dh0,
                            void* workspace, size_t workspace_bytes, void* stream) {
    SsmArgs a;
    if (gdr_status st = ssm_args(p, cu_seqlens, cu_seqlens != nullptr, &a)) return st;
    const int64_t e = element_size(p->io_dtype);
    const bool any = a.total > 0;
    if (gdr_status st = check({{cu_seqlens, 4, false}, {x, e, any}, {dt, e, any}, {A, 4, true}, {B, e, any}, {C, e, any},
                               {Dk, 4, false}, {z, e, false}, {dt_bias, 4, false}, {h0, 4, false}, {dy, e, any},
                               {dh_final, 4, false}, {dx, e, any}, {ddt, e, any}, {dA, 4, true}, {dB, e, any},
                               {dC, e, any}, {dDk, 4, false}, {dz, e, any && z}, {ddt_bias, 4, false}, {dh0, 4, false}}))
        return st;
    if (gdr_status st = check_workspace(workspace, workspace_bytes, ssm_backward_workspace(a))) return st;
    const SsmGrads g{dy, dh_final, dx, ddt, dA, dB, dC, dDk, dz, ddt_bias, dh0};
    return done(ssm_backward(a, ssm_tensors(p, x, dt, A, B, C, Dk, z, dt_bias, h0), g, (float*)workspace,
                             (cudaStream_t)stream),
                "ssm");
}

gdr_status gdr_ssm_step(const gdr_ssm_problem* p, const int32_t* slots, const void* x, const void* dt, const float* A,
                        const void* B, const void* C, const float* Dk, const void* z, const float* dt_bias, float* h,
                        void* y, void* stream) {
    if (!p) return GDR_ERR_NULL;
    gdr_ssm_problem one = *p;
    one.T = 1;
    SsmArgs a;
    if (gdr_status st = ssm_args(&one, nullptr, false, &a)) return st;
    if (p->pool < 1 || p->pool >= kMaxTokens || (!slots && p->n > p->pool)) return GDR_ERR_SHAPE;
    const int64_t e = element_size(p->io_dtype);
    if (gdr_status st = check({{slots, 4, false}, {x, e, true}, {dt, e, true}, {A, 4, true}, {B, e, true}, {C, e, true},
                               {Dk, 4, false}, {z, e, false}, {dt_bias, 4, false}, {h, 4, true}, {y, e, true}}))
        return st;
    return done(ssm_step(a, ssm_tensors(p, x, dt, A, B, C, Dk, z, dt_bias, nullptr), p->pool, slots, h, y,
                         (cudaStream_t)stream),
                "ssm_step");
}

}  // extern "C"
