// Internal declarations of the 8-bit operators (FP8 products, quantisation,
// norms); the public side is in include/dense_int8_matrix.h.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/dense_int8_matrix.h"

namespace gemm {

constexpr int kF8Block = 128;   // columns (or rows and columns) that share a scale

// One FP8 product, checked by the entry point.
struct F8Launch {
    const uint8_t* A;        // m x k, row pitch lda
    const uint8_t* Bt;       // n x k, row pitch ldb; GEMM_GROUP_ROWS: groups * n rows
    const float* a_scale;    // [kb][m]
    const float* b_scale;    // GEMM_SCALE_BLOCKS: [group][ceil(n / 128)][kb]; GEMM_SCALE_ROWS: [kb][b_rows]
    const int32_t* offsets;  // groups + 1 row offsets (grouped products)
    void* D;                 // m x n, row pitch ldd; GEMM_GROUP_K: groups of m rows
    int* err;                // device error word
    int64_t m, k, n, lda, ldb, ldd;
    int64_t rows_a, rows_b;  // rows of the whole A and Bt
    int groups, group_mode;
    int a_type, b_type, b_scale_mode;
    bool out_f32;
    int bm, bn, split_k;
    int num_sms, pairs;
};

// Two-SM tiles of 256 x bn (gemm_f8_tc2.cu).
cudaError_t launch_f8_tc2(const F8Launch& a, cudaStream_t stream);
// Tiles of bm (16, 32, 64, 128) rows x 128 columns of D, split_k CTAs each (gemm_f8_skinny.cu).
cudaError_t launch_f8_skinny(const F8Launch& a, cudaStream_t stream);

// ---- quantisation (quantize.cu) ----------------------------------------------
struct F8Quant {
    const void* X;
    int x_type;
    int64_t rows, cols, ldx;
    int f8_type;
    const int32_t* offsets;   // column form only; nullptr: one group of all rows
    int groups;
    int64_t kp;               // column form: padded columns of Q
    uint8_t* Q;
    int64_t ldq;
    float* scale;
    int num_sms;
};
cudaError_t launch_f8_quant_rows(const F8Quant& q, cudaStream_t stream);
cudaError_t launch_f8_quant_blocks(const F8Quant& q, cudaStream_t stream);
cudaError_t launch_f8_quant_cols(const F8Quant& q, cudaStream_t stream);

// ---- norms (norm.cu) -------------------------------------------------------------
struct NormFwd {
    const void *X, *R;
    const float* W;
    float eps;
    int x_type;
    int64_t rows, d, ldx, ldr, ldh, ldq;
    void* H;
    float* rstd;
    void* Q;        // e4m3, or int8 (to_i8)
    float* scale;   // [kb][rows], or [rows] (to_i8)
    bool to_i8;
    int num_sms;
};
cudaError_t launch_norm_fwd(const NormFwd& a, cudaStream_t stream);

struct NormBwd {
    const void *dY, *H, *dR;
    const float *W, *rstd;
    int x_type;
    int64_t rows, d, lddy, ldh, lddr, lddx;
    void* dX;
    float* dW;        // d sums, or nullptr
    float* partial;   // grid x d sums when grid > 1 (16-byte aligned)
    int grid;
    int num_sms;
    int* err;         // device error word
};
// CTAs of the backward kernel for the call's other fields; with more than one,
// dW needs grid * d floats of scratch.
int norm_bwd_grid(const NormBwd& a);
cudaError_t launch_norm_bwd(const NormBwd& a, cudaStream_t stream);

}  // namespace gemm
