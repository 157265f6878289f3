// Arguments and launchers of the operators in 8-bit blocks (norm.hip, blocks.hip): codes in e4m3
// (FN, largest value 448) with a binary32 scale for every 128 consecutive elements of a row of
// activations, and for every 128 x 128 elements of a matrix.
#pragma once

#include "coded.h"

namespace exl3 {

constexpr int kBlock = 128;                      // elements a scale serves along a row
constexpr float kCodeMax = 448.0f;               // the largest e4m3 value

__host__ __device__ inline int blocks_of(int width) { return (width + kBlock - 1) / kBlock; }

// Rows of activations as blocks: codes [n][ld], ld a multiple of 128, zero past the width;
// scales [blocks][lds], a row's scales lds apart, so that those of neighbouring rows are
// neighbours, as the product reads them.
struct BlockRowsArgs {
    uint8_t *q;
    float *scale;
    int64_t ld, lds;
};

// Matrices as blocks: codes [groups][rows][ld], scales [groups][blocks_of(rows)][blocks_of(cols)].
struct BlockWeightArgs {
    const uint8_t *q;
    const float *scale;
    int groups, rows, cols;
    int64_t ld;
};

// ---- norm.hip ----
struct NormArgs {
    const void *x, *residual;                    // residual: null for none
    int64_t ldx, ldr;
    const void *gain;
    bool gain32;                                 // binary32, else of the type of x
    float eps;
    int64_t n;
    int cols;
    void *y;                                     // null: blocks into q
    int64_t ldy;
    void *sum;                                   // with a residual: x + residual, or null
    int64_t ldsum;
    BlockRowsArgs q;
};
hipError_t launch_rms_norm(const NormArgs &a, bool bf16, int n_cu, hipStream_t stream);

struct NormBackwardArgs {
    const void *dy, *s, *ds;                     // ds: null for none
    int64_t lddy, lds, ldds;
    const void *gain;
    bool gain32;
    float eps;
    int64_t n;
    int cols;
    void *dx;
    int64_t lddx;
    void *dgain;                                 // of gain's type, or null
    float *part;                                 // [parts][cols]
    int parts;
};
int norm_backward_parts(int64_t n, int cols, int n_cu);
hipError_t launch_rms_norm_backward(const NormBackwardArgs &a, bool bf16, hipStream_t stream);

hipError_t launch_block_quantize(const void *x, int64_t ldx, int64_t n, int cols, bool bf16,
                                 const BlockRowsArgs &out, int n_cu, hipStream_t stream);

// dtype: EXL3_F32, EXL3_BF16 or EXL3_F16; w [rows][ldw].
hipError_t launch_block_quantize_weight(const void *w, int dtype, int64_t ldw, int rows, int cols,
                                        uint8_t *q, int64_t ldq, float *scale, hipStream_t stream);

// ---- blocks.hip ----
// y[n][out] = x W^T, or x W when transposed, for each group's rows; the rows of no group become
// zero.  x: codes of width cols (rows when transposed).
struct BlockProductArgs {
    BlockRowsArgs x;
    int64_t n;
    const int32_t *offsets;                      // null: one group of all rows
    bool transposed;
    void *y;
    int64_t ldy;
};
hipError_t launch_block_gemm(const BlockWeightArgs &w, const BlockProductArgs &a, bool bf16,
                             int n_cu, hipStream_t stream);

}  // namespace exl3
