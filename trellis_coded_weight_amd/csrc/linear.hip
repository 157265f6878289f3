// Products of few rows with coded weights, y = x W^T, on gfx950.
//
// W = diag(su) H_l (scale C) H_r diag(sv) with C the codes' levels, so
//   y = scale / had * su (H_l (C x')),   x' = H_r (sv x)
// (H here without its factor 1 / sqrt(had), which enters twice).  Three
// launches: x' (rotate_kernel), C x' from the codes (coded_rows_kernel), and
// the sum, the left transform and the factors (finish_kernel).
#include "coded.h"

namespace exl3 {

namespace {

// Butterflies of the natural-order Sylvester Hadamard over `had` consecutive
// values, E per lane: log2(E) stages in registers, the rest across lanes.
template <int E>
__device__ __forceinline__ void hadamard_lanes(float (&v)[E], int had) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int s = 1; s < E; s <<= 1)
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (!(i & s)) {
                const float a = v[i], b = v[i + s];
                v[i] = a + b;
                v[i + s] = a - b;
            }
    for (int m = 1; m * E < had; m <<= 1) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float o = __shfl_xor(v[i], m);
            v[i] = (lane & m) ? o - v[i] : v[i] + o;
        }
    }
}

// ---- x' ----
// Half a wave per row and unit of 256 columns, eight columns a lane.  x' is
// held in binary16, whose products with the levels (binary16 themselves) the
// matrix instruction sums in binary32.  The unit's scale is the power of two
// that takes its largest magnitude into [2^13, 2^14): rounding then costs
// 2^-12 of each value down to 2^-27 of the largest, whatever the range of the
// activations (bfloat16's is far wider than binary16's).  A unit with a NaN or
// an infinity becomes NaN throughout.
template <bool BF>
__global__ void __launch_bounds__(256)
rotate_kernel(const uint16_t *__restrict__ x, int64_t ldx, int64_t n, int cols, int had, int units,
              const float *__restrict__ sv, const int32_t *__restrict__ offsets, int groups,
              uint16_t *__restrict__ xh, float *__restrict__ xs) {
    const int lane = threadIdx.x & 63, pairs = (units + 1) / 2;
    const int64_t wave = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t row = wave / pairs;
    if (row >= n) return;
    if (offsets) {
        const int e = group_of_row(offsets, groups, row);
        sv += (size_t)(e < groups ? e : groups - 1) * cols;
    }
    const int unit = (int)(wave - row * pairs) * 2 + (lane >> 5);
    const int col = unit * kUnit + (lane & 31) * 8;
    const bool in = col < cols;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = in ? Act<BF>::load(x[row * ldx + col + i]) * sv[col + i] : 0.0f;
    hadamard_lanes(v, had);
    float big = 0.0f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        big = fmaxf(big, fabsf(v[i]));
        bad |= !(fabsf(v[i]) <= 3.402823466e38f);
    }
    for (int m = 1; m < 32; m <<= 1) {
        big = fmaxf(big, __shfl_xor(big, m));
        bad |= __shfl_xor((int)bad, m) != 0;
    }
    // exponent of the largest: big in [2^(ex - 127), 2^(ex - 126)); its scale
    // 2^(ex - 140), held in the normal range
    int ex = (int)(__builtin_bit_cast(uint32_t, big) >> 23);
    ex = ex < 14 ? 14 : ex;
    const float scale = __builtin_bit_cast(float, (uint32_t)(ex - 13) << 23);
    // 1 / scale = 2^(140 - ex), in two factors as it may pass the largest power
    const float up = __builtin_bit_cast(float, (uint32_t)(127 + (140 - ex) / 2) << 23);
    const float up2 = __builtin_bit_cast(float, (uint32_t)(127 + (140 - ex) - (140 - ex) / 2) << 23);
    if (!in) return;
    u32x4 out;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f16x2 h;
        h[0] = (_Float16)(v[2 * i] * up * up2);
        h[1] = (_Float16)(v[2 * i + 1] * up * up2);
        out[i] = bad ? 0x7E007E00u : __builtin_bit_cast(uint32_t, h);
    }
    *reinterpret_cast<u32x4 *>(xh + row * cols + col) = out;
    if ((lane & 31) == 0) xs[row * units + unit] = scale;
}

// ---- C x' ----
// A workgroup of eight waves per 16 rows of W, group and split; the waves take
// the split's units of 256 columns in turn, and their sums meet in shared
// memory.  A wave decodes 16 x 64 weights into the operands of two steps and
// uses them for NT tiles of 16 activation rows; x' comes from the caches.
template <int LV, int K, int NT>
__global__ void __launch_bounds__(512)
coded_rows_kernel(const uint32_t *__restrict__ packed, Levels lv, int rows, int cols, int Kr,
                  const int32_t *__restrict__ offsets, const uint16_t *__restrict__ xh,
                  const float *__restrict__ xs, int64_t n, int split,
                  float *__restrict__ part) {
    __shared__ f32x4 sums[8][NT][64];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int r = lane & 15, g = lane >> 4;
    const int row_tiles = rows / 16, units = (cols + kUnit - 1) / kUnit;
    const int rt = blockIdx.x % row_tiles, sp = blockIdx.x / row_tiles, e = blockIdx.y;
    int64_t lo, hi;
    group_rows(offsets, e, n, lo, hi);
    const int kk = K ? K : Kr;
    const uint32_t *wrow = packed + ((size_t)e * row_tiles + rt) * (size_t)(cols / 16) * (8 * kk);
    for (int64_t t0 = lo; t0 < hi; t0 += 16 * NT) {
        const uint16_t *xr[NT];
        const float *sr[NT];
        f32x4 total[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            int64_t tok = t0 + 16 * t + r;
            tok = tok < hi ? tok : hi - 1;     // a row past the end repeats the last, unstored
            xr[t] = xh + tok * cols;
            sr[t] = xs + tok * units;
            total[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        for (int u = sp * 8 + wv; u < units; u += 8 * split) {
            const int c0 = u * kUnit;
            uint32_t d[4][RowWords<K>::N];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (c0 + 64 * q < cols)
                    load_row<K>(wrow + (size_t)(c0 / 16 + 4 * q + g) * (8 * kk), r, d[q]);
            f32x4 acc[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (c0 + 64 * q >= cols) break;
                u32x4 w[2];
                decode_row<LV, K>(wrow + (size_t)(c0 / 16 + 4 * q + g) * (8 * kk), r, d[q], lv, w);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const u32x4 *xp =
                        reinterpret_cast<const u32x4 *>(xr[t] + c0 + 64 * q + 16 * g);
                    acc[t] = Act<false>::mfma(w[0], xp[0], acc[t]);
                    acc[t] = Act<false>::mfma(w[1], xp[1], acc[t]);
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float s = sr[t][u];
#pragma unroll
                for (int i = 0; i < 4; ++i) total[t][i] += s * acc[t][i];
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) sums[wv][t][lane] = total[t];
        __syncthreads();
        for (int i = threadIdx.x; i < NT * 64; i += 512) {
            const int t = i >> 6, l = i & 63;
            f32x4 a = sums[0][t][l];
#pragma unroll
            for (int w = 1; w < 8; ++w) a += sums[w][t][l];
            const int64_t tok = t0 + 16 * t + (l & 15);
            if (tok < hi)
                *reinterpret_cast<f32x4 *>(part + ((size_t)sp * n + tok) * rows + rt * 16 +
                                           4 * (l >> 4)) = a;
        }
        __syncthreads();
    }
}

// ---- y ----
// A wave per row of y and 256 of its columns, four a lane.
template <bool BF>
__global__ void __launch_bounds__(256)
finish_kernel(const float *__restrict__ part, int split, int64_t n, int rows, int had,
              const float *__restrict__ scale, const float *__restrict__ su,
              const int32_t *__restrict__ offsets, int groups, AdapterArgs ad,
              const uint16_t *__restrict__ v, uint16_t *__restrict__ y, int64_t ldy) {
    const int lane = threadIdx.x & 63, blocks = (rows + 255) / 256;
    const int64_t wave = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t tok = wave / blocks;
    if (tok >= n) return;
    const int row = (int)(wave - tok * blocks) * 256 + lane * 4;
    const bool in = row < rows;
    int e = 0;
    if (offsets) {
        e = group_of_row(offsets, groups, tok);
        if (e >= groups || tok < offsets[0]) {
            if (in)
                for (int i = 0; i < 4; ++i) y[tok * ldy + row + i] = 0;
            return;
        }
    }
    float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (in)
        for (int s = 0; s < split; ++s) {
            const f32x4 p = *reinterpret_cast<const f32x4 *>(part + ((size_t)s * n + tok) * rows + row);
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] += p[i];
        }
    hadamard_lanes(a, had);
    if (!in) return;
    const float f = scale[e] / (float)had;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] *= f * su[(size_t)e * rows + row + i];
    if (v) {
        const int id = ad.ids[tok];
        if (id >= 0 && id < ad.count) {
            const uint16_t *b = static_cast<const uint16_t *>(ad.b) +
                                ((size_t)id * rows + row) * ad.rank;
            const uint16_t *vt = v + tok * ad.rank_pad;
            for (int k = 0; k < ad.rank; ++k) {
                const float vk = Act<BF>::load(vt[k]);
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] += vk * Act<BF>::load(b[i * ad.rank + k]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) y[tok * ldy + row + i] = Act<BF>::store(a[i]);
}

template <int LV, int K>
hipError_t coded_rows_t(const WeightArgs &w, const int32_t *offsets, const uint16_t *xh,
                        const float *xs, int64_t n, int split, int tiles, float *part,
                        hipStream_t stream) {
    const dim3 grid((unsigned)(w.rows / 16 * split), (unsigned)w.groups);
#define EXL3_ROWS(NT)                                                                        \
    hipLaunchKernelGGL((coded_rows_kernel<LV, K, NT>), grid, dim3(512), 0, stream, w.packed, \
                       w.lv, w.rows, w.cols, w.K, offsets, xh, xs, n, split, part)
    if (tiles <= 1)
        EXL3_ROWS(1);
    else if (tiles <= 2)
        EXL3_ROWS(2);
    else
        EXL3_ROWS(4);
#undef EXL3_ROWS
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rotate(const WeightArgs &w, const int32_t *offsets, const void *x, int64_t ldx,
                         int64_t n, bool bf16, uint16_t *xh, float *xs, hipStream_t stream) {
    const int units = (w.cols + kUnit - 1) / kUnit;
    const unsigned grid = (unsigned)((n * ((units + 1) / 2) + 3) / 4);
    const uint16_t *xx = static_cast<const uint16_t *>(x);
    if (bf16)
        hipLaunchKernelGGL((rotate_kernel<true>), dim3(grid), dim3(256), 0, stream, xx, ldx, n,
                           w.cols, w.had, units, w.sv, offsets, w.groups, xh, xs);
    else
        hipLaunchKernelGGL((rotate_kernel<false>), dim3(grid), dim3(256), 0, stream, xx, ldx, n,
                           w.cols, w.had, units, w.sv, offsets, w.groups, xh, xs);
    return hipGetLastError();
}

hipError_t launch_coded_rows(const WeightArgs &w, const int32_t *offsets, const uint16_t *xh,
                             const float *xs, int64_t n, int split, int tiles, float *part,
                             hipStream_t stream) {
#define EXL3_ROWS_K(LV, KK) \
    case KK: return coded_rows_t<LV, KK>(w, offsets, xh, xs, n, split, tiles, part, stream)
    if (w.lv_kind == kLevelsMul1)
        switch (w.K) {
            EXL3_ROWS_K(kLevelsMul1, 1);
            EXL3_ROWS_K(kLevelsMul1, 2);
            EXL3_ROWS_K(kLevelsMul1, 3);
            EXL3_ROWS_K(kLevelsMul1, 4);
        }
    else if (w.lv_kind == kLevelsHalves)
        switch (w.K) {
            EXL3_ROWS_K(kLevelsHalves, 1);
            EXL3_ROWS_K(kLevelsHalves, 2);
            EXL3_ROWS_K(kLevelsHalves, 3);
            EXL3_ROWS_K(kLevelsHalves, 4);
        }
#undef EXL3_ROWS_K
    return coded_rows_t<kLevelsTable, 0>(w, offsets, xh, xs, n, split, tiles, part, stream);
}

hipError_t launch_finish(const WeightArgs &w, const int32_t *offsets, const float *part, int split,
                         int64_t n, bool bf16, const AdapterArgs *ad, const uint16_t *v, void *y,
                         int64_t ldy, hipStream_t stream) {
    const unsigned grid = (unsigned)((n * ((w.rows + 255) / 256) + 3) / 4);
    const AdapterArgs args = ad ? *ad : AdapterArgs{};
    uint16_t *yy = static_cast<uint16_t *>(y);
    if (bf16)
        hipLaunchKernelGGL((finish_kernel<true>), dim3(grid), dim3(256), 0, stream, part, split, n,
                           w.rows, w.had, w.scale, w.su, offsets, w.groups, args, v, yy, ldy);
    else
        hipLaunchKernelGGL((finish_kernel<false>), dim3(grid), dim3(256), 0, stream, part, split,
                           n, w.rows, w.had, w.scale, w.su, offsets, w.groups, args, v, yy, ldy);
    return hipGetLastError();
}

}  // namespace exl3
