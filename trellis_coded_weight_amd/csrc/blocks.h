// Arguments and launchers of the operators in 8-bit blocks (norm.hip, blocks.hip): codes in e4m3
// (FN, largest value 448) with a binary32 scale for every 128 consecutive elements of a row of
// activations, and for every 128 x 128 elements of a matrix.
#pragma once

#include <float.h>

#include "block_forms.h"
#include "coded.h"

namespace exl3 {

constexpr float kCodeMax = 448.0f;               // the largest e4m3 value
constexpr size_t kOwnBytes = 48 << 10;           // shared memory for rows a workgroup writes as blocks

// ---- device side: 16-bit rows and their codes ----
constexpr int kWide = 8;                         // consecutive elements a lane takes at a time

// Eight consecutive 16-bit elements, `valid` of them there; the rest are zero.
__device__ __forceinline__ u32x4 load8(const uint16_t *p, int valid) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (valid >= kWide) return *reinterpret_cast<const u32x4u *>(p);
    for (int i = 0; i < valid; ++i) v[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    return v;
}
__device__ __forceinline__ void store8(uint16_t *p, u32x4 v, int valid) {
    if (valid >= kWide) {
        *reinterpret_cast<u32x4u *>(p) = v;
        return;
    }
    for (int i = 0; i < valid; ++i) p[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
}
template <bool BF>
__device__ __forceinline__ void widen(u32x4 v, float (&f)[kWide]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = Act<BF>::load((uint16_t)v[i]);
        f[2 * i + 1] = Act<BF>::load((uint16_t)(v[i] >> 16));
    }
}
template <bool BF>
__device__ __forceinline__ u32x4 narrow(const float (&f)[kWide]) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = Act<BF>::store2(f[2 * i], f[2 * i + 1]);
    return v;
}

// The scale of a block whose largest magnitude has these bits; what its values are multiplied by
// first (2^64 for tiny blocks, else one), the scale times that, and the inverse of the latter.  The
// scale stays in the normal range, so that the inverse does too.  NaN where the block holds an
// infinity or a NaN: magnitudes compare as integers, which keeps a NaN.
struct CodeScale {
    float scale, lift, lifted, inverse;
};
__device__ __forceinline__ CodeScale code_scale(uint32_t big) {
    CodeScale s;
    s.scale = __builtin_bit_cast(float, big) / kCodeMax;
    s.scale = s.scale < FLT_MIN ? FLT_MIN : s.scale;
    if (big >= 0x7F800000u) s.scale = __builtin_bit_cast(float, 0x7FC00000u);
    s.lift = s.scale < 0x1p-60f ? 0x1p64f : 1.0f;
    s.lifted = s.scale * s.lift;
    s.inverse = 1.0f / s.lifted;
    return s;
}
// v / scale rounded to binary32 as a division does: the product with the correctly rounded
// inverse is at most one unit off, and the remainder brings it to the nearest (taken with this
// sign, it leaves a zero's sign alone).  The remainder is exact, as the lift keeps it out of the
// subnormal numbers for every value that has a code other than zero (its last place, 2^-47 of v or
// less, stays above 2^-149 for v from 2^-102 on; codes end at 2^-10 of the scale).
// The instruction then rounds to e4m3, ties to even; at 448 (1 + 2^-23) nothing overflows.
__device__ __forceinline__ float quotient(float v, const CodeScale &s) {
    v *= s.lift;
    const float q = v * s.inverse;
    return __builtin_fmaf(-__builtin_fmaf(q, s.lifted, -v), s.inverse, q);
}
__device__ __forceinline__ u32x2 to_codes(const float (&f)[kWide], const CodeScale &s) {
    u32x2 o;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(f[4 * h], s), quotient(f[4 * h + 1], s), 0,
                                                false);
        v = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(f[4 * h + 2], s), quotient(f[4 * h + 3], s), v,
                                            true);
        o[h] = (uint32_t)v;
    }
    return o;
}
// Codes with those past the first `valid` zero, as behind a row's end also in a block of NaN.
__device__ __forceinline__ u32x2 first_codes(u32x2 codes, int valid) {
    if (valid < kWide) {
        const uint64_t keep = valid > 0 ? (1ull << 8 * valid) - 1 : 0;
        codes[0] &= (uint32_t)keep;
        codes[1] &= (uint32_t)(keep >> 32);
    }
    return codes;
}
__device__ __forceinline__ uint32_t magnitude(float v) {
    return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu;
}
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t largest8(const float (&f)[kWide]) {
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < kWide; ++i) big = larger(big, magnitude(f[i]));
    return big;
}
// Over 16 neighbouring lanes, a block's columns.
__device__ __forceinline__ uint32_t largest_of_block(uint32_t big) {
    float f = __builtin_bit_cast(float, big);
    big = larger(big, __builtin_bit_cast(uint32_t, lane_xor<1>(f)));
    f = __builtin_bit_cast(float, big);
    big = larger(big, __builtin_bit_cast(uint32_t, lane_xor<2>(f)));
    f = __builtin_bit_cast(float, big);
    big = larger(big, __builtin_bit_cast(uint32_t, lane_xor<4>(f)));
    f = __builtin_bit_cast(float, big);
    return larger(big, __builtin_bit_cast(uint32_t, lane_xor<8>(f)));
}

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
hipError_t launch_rms_norm(const NormArgs &a, bool bf16, hipStream_t stream);

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
                                 const BlockRowsArgs &out, hipStream_t stream);

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
    const void *x16;                             // 16-bit rows in place of x (launch_block_rows)
    int64_t ldx16;
};
// Few rows a group, not transposed; x or x16.
hipError_t launch_block_rows(const BlockWeightArgs &w, const BlockProductArgs &a, bool bf16,
                             hipStream_t stream);
// form: one of the tiles.
hipError_t launch_block_gemm(const BlockWeightArgs &w, const BlockProductArgs &a, BlockForm form,
                             bool bf16, hipStream_t stream);

}  // namespace exl3
