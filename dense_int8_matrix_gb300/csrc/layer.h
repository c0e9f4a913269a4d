// Internal declarations of the bfloat16 layer's operators (products with an
// epilogue, activation gradient, layer norm, balance loss); the public side is
// in include/dense_int8_matrix.h.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/dense_int8_matrix.h"

namespace gemm {

// ---- products ------------------------------------------------------------------
// One product, checked by the entry point: operands 16-byte aligned, pitches
// multiples of 8.
struct LinearLaunch {
    const void *A, *B;      // bfloat16, as GEMM_FORM_* says
    const float* bias;      // n floats or nullptr
    const void* R;          // residual, type and shape of D, or nullptr
    void* Z;                // bfloat16 m x n: written, or read (grad); or nullptr
    void* D;
    int* err;               // device error word
    int64_t m, k, n, lda, ldb, ldd, ldr, ldz;
    int form;
    int act;                // GEMM_ACT_* without GEMM_ACT_GRADIENT
    bool grad, out_f32;
    int bm, bn, split_k;
    int num_sms, pairs;
};
// Two-SM tiles of 256 x bn (gemm_linear_tc2.cu).
cudaError_t launch_linear_tc2(const LinearLaunch& a, cudaStream_t stream);
// Tiles of bm (16, 32, 64, 128; GEMM_FORM_TN 64, 128) rows x 128 columns, split_k CTAs each (gemm_linear_skinny.cu).
cudaError_t launch_linear_skinny(const LinearLaunch& a, cudaStream_t stream);

// Copies bfloat16 matrices of any address and pitch to rows that are 16-byte
// aligned (dst, pitch a multiple of 8); rows == 0: none.
struct Repitch {
    const void* src;
    int64_t ld;
    void* dst;
    int64_t pitch, rows, cols;
};
cudaError_t launch_repitch(const Repitch& a, const Repitch& b, int num_sms, cudaStream_t stream);

// ---- sums over rows ------------------------------------------------------------
// out[j] = sum over the parts of partial[part][j], in order (norm.cu).
cudaError_t launch_column_sums(const float* partial, int parts, int64_t d, float* out, cudaStream_t stream);

// ---- gradient of an activation and its bias (activation.cu) --------------------
struct ActBwd {
    const void *dY, *Z;
    void* dZ;
    float* dbias;     // cols sums, or nullptr
    float* partial;   // clusters x cols sums when there are several clusters
    int64_t rows, cols, lddy, ldz, lddz;
    int act;
    int parts;        // row ranges
    int num_sms;
};
int act_bwd_parts(const ActBwd& a);
int act_bwd_clusters(const ActBwd& a);   // of row ranges, once parts is set
cudaError_t launch_act_bwd(const ActBwd& a, cudaStream_t stream);

// ---- layer norm (layer_norm.cu, layer_norm_bwd.cu) ------------------------------------------------
struct LayerNormFwd {
    const void *X, *R;
    const float *W, *bias;
    float eps;
    int x_type, y_type;
    int64_t rows, d, ldx, ldr, ldh, ldy;
    void *H, *Y;
    float *mean, *rstd;
    int num_sms;
    int* err;            // device error word
};
cudaError_t launch_layer_norm_fwd(const LayerNormFwd& a, cudaStream_t stream);

struct LayerNormBwd {
    const void *dY, *H, *dR;
    const float *W, *mean, *rstd;
    int x_type, y_type;
    int64_t rows, d, lddy, ldh, lddr, lddx;
    void* dX;
    float *dW, *dbias;   // d sums each, or nullptr
    float* partial;      // 2 x parts x d sums (dW's, then dbias's) when parts > 1
    int parts;
    int num_sms;
    int* err;
};
int layer_norm_bwd_parts(const LayerNormBwd& a);
// Number of kernels it launches is written to *launches.
cudaError_t launch_layer_norm_bwd(const LayerNormBwd& a, cudaStream_t stream, int* launches);

// ---- balance loss (balance.cu) -------------------------------------------------
struct Balance {
    const void* X;
    int x_type;
    int64_t rows, ldx;
    int experts, top_k;
    const int32_t* index;
    float coef;
    int32_t *counts, *offsets, *used;
    float *lse, *probs, *loss;
    float* partial_p;     // parts x experts
    int32_t* partial_c;   // parts x (experts + 1): counts, and behind them the used rows
    int parts;            // clusters of CTAs; with more than one, scratch for their sums
    int num_sms;
};
int balance_parts(const Balance& a);
cudaError_t launch_balance(const Balance& a, cudaStream_t stream, int* launches);

struct BalanceBwd {
    const void *X, *dR;
    void* dX;
    int x_type;
    int64_t rows, ldx, lddr, lddx;
    int experts;
    const float* lse;
    const int32_t *counts, *used;
    float coef;
    const float* dloss;
    int num_sms;
};
cudaError_t launch_balance_bwd(const BalanceBwd& a, cudaStream_t stream);

}  // namespace gemm
