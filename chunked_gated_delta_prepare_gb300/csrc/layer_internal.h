// Internal interface between the C ABI of the layer operators (layer_api.cpp) and their kernel files.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gdr.h"

namespace gdr {

// Name of the kernel variant a call launched (gdr_last_variant; kept in gdr_api.cpp).
void set_last_variant(const char* name);

namespace layer {

// A tensor of rows: row i starts `ld` elements after row i - 1.
struct RowTensor {
    const void* p;
    int64_t ld;
    bool vec;      // every row starts on a 16-byte boundary
};

constexpr int kSms = 152;   // GB300

// ---- norm.cu
constexpr int64_t kNormMaxD = 32768;
struct NormArgs {
    int64_t rows;
    int D;
    int group;     // columns of a scale, 0: the row
    float eps;
    int io;        // gdr_dtype
};
cudaError_t norm_forward(const NormArgs& a, RowTensor x, RowTensor res, const void* w, void* y, void* r, void* y8,
                         float* scales, cudaStream_t s);
// Rows of partial sums of dw [rows, D] that norm_backward writes and adds up.
int64_t norm_partial_rows(const NormArgs& a);
cudaError_t norm_backward(const NormArgs& a, const void* dy, const void* r, const void* w, const void* dr, void* dx,
                          float* dw, float* partial, cudaStream_t s);

// Column sums of in[0..rows), row i at i * ld, in an order that depends on the sizes alone: the first `cols` columns
// go to out, the `cols2` after them to out2.
cudaError_t column_sum(const float* in, int64_t rows, int64_t ld, int64_t cols, float* out, int64_t cols2, float* out2,
                       cudaStream_t s);

// ---- conv.cu
struct ConvArgs {
    int64_t n, T, total;   // cu: total tokens on the packed axis; else n * T
    const int* cu;
    int64_t D;
    int W;
    int io;                // gdr_dtype
    bool silu;
};
constexpr int kConvMinW = 2, kConvMaxW = 4;
cudaError_t conv_forward(const ConvArgs& a, RowTensor x, const void* w, const void* b, const void* state, void* y,
                         void* state_out, cudaStream_t s);
// Rows of partial sums [D * W + D] of dw and db that conv_backward writes and adds up.
int64_t conv_partial_rows(const ConvArgs& a);
cudaError_t conv_backward(const ConvArgs& a, RowTensor x, const void* w, const void* b, const void* state,
                          const void* dy, const void* d_state_out, void* dx, float* dw, float* db, void* d_state,
                          float* partial, cudaStream_t s);
cudaError_t conv_step(const ConvArgs& a, int64_t pool, const int* slots, RowTensor x, const void* w, const void* b,
                      void* state, void* y, cudaStream_t s);

// ---- delta_step.cu
struct DeltaStepArgs {
    int64_t B, pool;
    int H, HV, K, V;
    int64_t q_ld, k_ld, v_ld;   // elements between the rows of a batch
    float scale;
    int io;                     // gdr_dtype
    bool per_k;
};
cudaError_t delta_step(const DeltaStepArgs& a, const int* slots, const void* q, const void* k, const void* v,
                       const float* g, const void* beta, float* h, void* o, cudaStream_t s);

// ---- ssm.cu
constexpr int kSsmMaxN = 64;
constexpr int kSsmMinWidth = 16;   // channels of the smallest block: of the step's and the gradient's at more than 32 states
struct SsmArgs {
    int64_t n, T, total;   // cu: total tokens on the packed axis; else n * T
    const int* cu;
    int D, N, G;
    int io;                // gdr_dtype
    bool softplus;
};
struct SsmTensors {
    RowTensor x, dt, z, B, C;
    const float *A, *bias, *Dk, *h0;
};
size_t ssm_forward_workspace(const SsmArgs& a);
cudaError_t ssm_forward(const SsmArgs& a, const SsmTensors& t, void* y, float* h_final, float* workspace,
                        cudaStream_t s);
cudaError_t ssm_step(const SsmArgs& a, const SsmTensors& t, int64_t pool, const int* slots, float* h, void* y,
                     cudaStream_t s);

// ---- ssm_backward.cu
struct SsmGrads {
    const void* dy;
    const float* dh_final;
    void *dx, *ddt;
    float* dA;
    void *dB, *dC;
    float* dDk;
    void* dz;
    float *dbias, *dh0;
};
size_t ssm_backward_workspace(const SsmArgs& a);
cudaError_t ssm_backward(const SsmArgs& a, const SsmTensors& t, const SsmGrads& g, float* workspace, cudaStream_t s);

// ---- lru.cu, lru_backward.cu
constexpr int kLruKept = 128;      // tokens from one kept state to the next
struct LruArgs {
    int64_t n, T, total;   // cu: total tokens on the packed axis; else n * T
    const int* cu;
    int D;
    int io;                // gdr_dtype
    float c;
};
struct LruTensors {
    RowTensor x, r, i;     // i.p nullptr: no input gate
    const float *lam, *h0; // lam nullptr: no rates
};
struct LruGrads {
    const void* dy;
    const float* dh_final;
    void *dx, *dr, *di;
    float *dlam, *dh0;
};
int64_t lru_tiles(const LruArgs& a);      // rows of the kept states
// y, h_final and kept may each be nullptr.
size_t lru_forward_workspace(const LruArgs& a);
cudaError_t lru_forward(const LruArgs& a, const LruTensors& t, void* y, float* h_final, float* kept, void* workspace,
                        cudaStream_t s);
size_t lru_backward_workspace(const LruArgs& a, bool kept);
cudaError_t lru_backward(const LruArgs& a, const LruTensors& t, const LruGrads& g, const float* kept, void* workspace,
                         cudaStream_t s);
cudaError_t lru_step(const LruArgs& a, const LruTensors& t, int64_t pool, const int* slots, float* h, void* y,
                     cudaStream_t s);

// ---- layer_norm.cu (NormArgs::group is not used)
cudaError_t layernorm_forward(const NormArgs& a, RowTensor x, RowTensor res, const void* w, const void* b, void* y,
                              void* r, cudaStream_t s);
// Rows of partial sums [2 D] of dw and db that layernorm_backward writes and adds up.
int64_t layernorm_partial_rows(const NormArgs& a);
cudaError_t layernorm_backward(const NormArgs& a, const void* dy, const void* r, const void* w, const void* dr, void* dx,
                               float* dw, float* db, float* partial, cudaStream_t s);

// ---- gated_norm.cu
constexpr int64_t kGatedNormMaxV = 8192;
struct GatedNormArgs {
    int64_t tokens;
    int H, V;
    float eps;
    int io;                // gdr_dtype
    bool silu, per_head;
};
cudaError_t gated_norm_forward(const GatedNormArgs& a, RowTensor x, RowTensor z, const void* w, void* y, cudaStream_t s);
// Rows of partial sums [V] of dw that gated_norm_backward writes and adds up.
int64_t gated_norm_partial_rows(const GatedNormArgs& a);
cudaError_t gated_norm_backward(const GatedNormArgs& a, const void* dy, RowTensor x, RowTensor z, const void* w, void* dx,
                                void* dz, float* dw, float* partial, cudaStream_t s);

}  // namespace layer
}  // namespace gdr
