// Products of many rows with coded weights on gfx950: the weights written once
// in the activations' type and their own domain (dense_kernel), then a matrix
// product (gemm_kernel).  Both directions, y = x W^T and y = x W, contract over
// consecutive elements: for the second the weights are written transposed.
#include "coded.h"

namespace exl3 {

namespace {

__device__ __forceinline__ uint32_t parity16(uint32_t v) { return __popc(v) & 1u; }

// ---- dense weights ----
// A workgroup per HB x HB block of W (HB: the Hadamard block), a wave per 16
// rows and then per 16 columns.  Both transforms run on the matrix units: the
// levels are exact in binary16 and the transform's entries are +-1.
//   1. The wave decodes 16 x 64 levels into operands (coded.h) and multiplies
//      by H_64 over their columns, an operand made of signs: entry (c, n) is
//      (-1)^popcount(c & n); for HB = 128 the halves' sum and difference
//      follow.
//   2. The result, sums of HB levels, is rounded to binary16 (2^-12 of each,
//      below the final rounding to binary16 or bfloat16) and passes through
//      shared memory column by column.
//   3. The wave multiplies 16 columns by H_HB over the rows, then the scale,
//      su and sv in binary32, and rounds once to the activations' type.
// Row-major and transposed output differ in the order of step 3's operands:
// either way a lane holds four consecutive elements of the output.
template <int LV, int K, int HB, bool BF, bool TR>
__global__ void __launch_bounds__(HB * 4)
dense_kernel(const uint32_t *__restrict__ packed, Levels lv, int rows, int cols, int Kr,
             const float *__restrict__ scale, const float *__restrict__ su,
             const float *__restrict__ sv, const int32_t *__restrict__ offsets, int64_t n, int g0,
             uint16_t *__restrict__ dense) {
    constexpr int kPitch = HB * 2 + 16;          // bytes a column of the block takes in LDS
    __shared__ __align__(16) char mid[HB * kPitch];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int r = lane & 15, g = lane >> 4;
    const int e = g0 + blockIdx.y, blocks = cols / HB;
    const int br = blockIdx.x / blocks, bc = blockIdx.x % blocks;
    int64_t lo, hi;
    group_rows(offsets, e, n, lo, hi);
    if (lo >= hi) return;                        // no row uses this group
    const int kk = K ? K : Kr;
    const int rt = br * (HB / 16) + wv;
    const uint32_t *tiles = packed + (((size_t)e * (rows / 16) + rt) * (cols / 16) +
                                      (size_t)bc * (HB / 16) + g) * (8 * kk);
    f32x4 sum[HB / 16];
    uint32_t d[HB / 64][RowWords<K>::N];
#pragma unroll
    for (int q = 0; q < HB / 64; ++q) load_row<K>(tiles + (size_t)(4 * q) * (8 * kk), r, d[q]);
#pragma unroll
    for (int q = 0; q < HB / 64; ++q) {
        u32x4 w[2];
        decode_row<LV, K>(tiles + (size_t)(4 * q) * (8 * kk), r, d[q], lv, w);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            f32x4 p = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                // signs of H_64 at rows 16 g + 8 s + j, column 16 t + r
                const uint32_t flip = parity16(g & t);
                u32x4 h;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t a = parity16((8 * s + 2 * j) & r) ^ flip;
                    const uint32_t b = parity16((8 * s + 2 * j + 1) & r) ^ flip;
                    h[j] = 0x3C003C00u | (a << 15) | (b << 31);
                }
                p = Act<false>::mfma(w[s], h, p);
            }
            if (q == 0) {
                sum[t] = p;
            } else {
                sum[(4 + t) % (HB / 16)] = sum[t] - p;
                sum[t] = sum[t] + p;
            }
        }
    }
    // column 16 t + r, rows 16 wv + 4 g .. + 3
#pragma unroll
    for (int t = 0; t < HB / 16; ++t) {
        f16x2 a, b;
        a[0] = (_Float16)sum[t][0];
        a[1] = (_Float16)sum[t][1];
        b[0] = (_Float16)sum[t][2];
        b[1] = (_Float16)sum[t][3];
        uint2 o;
        o.x = __builtin_bit_cast(uint32_t, a);
        o.y = __builtin_bit_cast(uint32_t, b);
        *reinterpret_cast<uint2 *>(mid + (16 * t + r) * kPitch + (16 * wv + 4 * g) * 2) = o;
    }
    __syncthreads();
    u32x4 m[HB / 32];
#pragma unroll
    for (int p = 0; p < HB / 32; ++p)
        m[p] = *reinterpret_cast<const u32x4 *>(mid + (16 * wv + r) * kPitch + (32 * p + 8 * g) * 2);
    const float f = scale[e] / (float)HB;
    const float *su_b = su + (size_t)e * rows + (size_t)br * HB;
    const float *sv_b = sv + (size_t)e * cols + (size_t)bc * HB;
    uint16_t *out = dense + (size_t)blockIdx.y * rows * cols;
#pragma unroll
    for (int t = 0; t < HB / 16; ++t) {
        f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int p = 0; p < HB / 32; ++p) {
            // signs of H_HB at row 16 t + r, rows 32 p + 8 g + j
            const uint32_t flip = parity16(t & (2 * p + (g >> 1)));
            u32x4 h;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t a = parity16(r & (8 * (g & 1) + 2 * j)) ^ flip;
                const uint32_t b = parity16(r & (8 * (g & 1) + 2 * j + 1)) ^ flip;
                h[j] = 0x3C003C00u | (a << 15) | (b << 31);
            }
            z = TR ? Act<false>::mfma(h, m[p], z) : Act<false>::mfma(m[p], h, z);
        }
        // transposed: column 16 wv + r, rows 16 t + 4 g ..; else row 16 t + r,
        // columns 16 wv + 4 g ..
        const int row = TR ? 16 * t + 4 * g : 16 * t + r, col = TR ? 16 * wv + r : 16 * wv + 4 * g;
        uint2 o;
        uint16_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q[i] = Act<BF>::store(z[i] * (f * su_b[TR ? row + i : row] * sv_b[TR ? col : col + i]));
        o.x = q[0] | ((uint32_t)q[1] << 16);
        o.y = q[2] | ((uint32_t)q[3] << 16);
        const size_t at = TR ? ((size_t)bc * HB + col) * rows + (size_t)br * HB + row
                             : ((size_t)br * HB + row) * cols + (size_t)bc * HB + col;
        *reinterpret_cast<uint2 *>(out + at) = o;
    }
}

// ---- matrix product ----
// y[n][m] = x[n][k] w[m][k]^T: the weights are the instruction's first operand
// and the rows of x its second, so a lane's four results are consecutive
// elements of one row of y.  A workgroup computes BM columns of y by BN rows;
// 64 of k at a time pass through two buffers in shared memory, the next ones
// loaded straight into it while these are used.  A load writes a wave's 64
// pieces of 16 bytes in lane order, so the swizzle that spreads a column of
// pieces over the banks is in which piece each lane fetches: piece s of row r
// holds k piece s ^ (r & 7).
template <int BM, int BN, int WM, int WN, bool BF>
__global__ void __launch_bounds__(64 * WM * WN)
gemm_kernel(const uint16_t *__restrict__ x, int64_t ldx, const uint16_t *__restrict__ w, int64_t n,
            int m, int k, const int32_t *__restrict__ offsets, int g0, int ng, int m_tiles,
            int total, AdapterArgs ad, const uint16_t *__restrict__ ad_b,
            const uint16_t *__restrict__ v, uint16_t *__restrict__ y, int64_t ldy) {
    constexpr int kThreads = 64 * WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
    constexpr int kPieces = (BM + BN) * 8 / kThreads;     // 16-byte pieces a thread loads
    __shared__ __align__(16) uint16_t buf[2][(BM + BN) * 64];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int r = lane & 15, g = lane >> 4, wm = wv % WM, wn = wv / WM;
    // consecutive workgroups go to different dies: give each die a run of tiles
    int id = blockIdx.x;
    {
        const int per = total / 8, rest = total % 8, die = id % 8;
        id = die * per + (die < rest ? die : rest) + id / 8;
    }
    const int mt = id % m_tiles;
    int nt = id / m_tiles, e = 0;
    int64_t lo = 0, hi = n;
    if (offsets) {
        // the group that holds the nt-th tile of rows, groups in order
        int before = 0;
        e = -1;
        for (int j = 0; j < ng; j += 64) {
            int64_t a = 0, b = 0;
            if (j + lane < ng) group_rows(offsets, g0 + j + lane, n, a, b);
            int sum = b > a ? (int)((b - a + BN - 1) / BN) : 0;
#pragma unroll
            for (int s = 1; s < 64; s <<= 1) {
                const int o = __shfl_up(sum, s);
                if (lane >= s) sum += o;
            }
            const uint64_t past = __ballot(before + sum > nt);
            if (past) {
                const int l = __ffsll((unsigned long long)past) - 1;
                const int prev = l ? __shfl(sum, l - 1) : 0;
                e = j + l;
                nt -= before + prev;
                break;
            }
            before += __shfl(sum, 63);
        }
        if (e < 0) return;                   // fewer tiles than the bound allows
        group_rows(offsets, g0 + e, n, lo, hi);
    }
    const int64_t row0 = lo + (int64_t)nt * BN;
    const uint16_t *wg = w + (size_t)e * m * k;

    const uint16_t *src[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const int piece = i * kThreads + threadIdx.x, row = piece >> 3;
        const int kp = (piece & 7) ^ (row & 7);
        if (row < BM) {
            int mr = mt * BM + row;
            mr = mr < m ? mr : m - 1;        // past the edge: repeats, not stored
            src[i] = wg + (size_t)mr * k + kp * 8;
        } else {
            int64_t xr = row0 + row - BM;
            xr = xr < hi ? xr : hi - 1;
            src[i] = x + xr * ldx + kp * 8;
        }
    }
    auto load = [&](int b) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            __builtin_amdgcn_global_load_lds(
                (const __attribute__((address_space(1))) void *)src[i],
                (__attribute__((address_space(3))) void *)(&buf[b][(i * kThreads + wv * 64) * 8]),
                16, 0, 0);
            src[i] += 64;
        }
    };
    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int steps = k / 64;
    load(0);
    for (int s = 0; s < steps; ++s) {
        __syncthreads();                     // this step's loads have landed, the other buffer is free
        if (s + 1 < steps) load((s + 1) & 1);
        const uint16_t *ba = buf[s & 1] + (size_t)(wm * (BM / WM)) * 64;
        const uint16_t *bb = buf[s & 1] + (size_t)(BM + wn * (BN / WN)) * 64;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int at = (((4 * h + g) ^ (r & 7)) * 8);
            u32x4 a[TM], b[TN];
#pragma unroll
            for (int i = 0; i < TM; ++i)
                a[i] = *reinterpret_cast<const u32x4 *>(ba + (16 * i + r) * 64 + at);
#pragma unroll
            for (int j = 0; j < TN; ++j)
                b[j] = *reinterpret_cast<const u32x4 *>(bb + (16 * j + r) * 64 + at);
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = Act<BF>::mfma(a[i], b[j], acc[i][j]);
        }
    }
    const int m0 = mt * BM + wm * (BM / WM);
    const int64_t t0 = row0 + wn * (BN / WN);
    if (v) {
        // v b^T of each adapter that some row of the wave has, in ascending
        // order; its result is added where the row's adapter is this one, so
        // nothing of another adapter's values reaches a row
        int idj[TN];
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int64_t tok = t0 + 16 * j + r;
            const int id2 = tok < hi ? ad.ids[tok] : -1;
            idj[j] = id2 >= 0 && id2 < ad.count ? id2 : 0x7FFFFFFF;
        }
        int last = -1;
        for (;;) {
            int next = 0x7FFFFFFF;
#pragma unroll
            for (int j = 0; j < TN; ++j) next = idj[j] > last && idj[j] < next ? idj[j] : next;
            for (int s = 1; s < 16; s <<= 1) {
                const int o = __shfl_xor(next, s);
                next = o < next ? o : next;
            }
            next = __builtin_amdgcn_readfirstlane(next);
            if (next == 0x7FFFFFFF) break;
            last = next;
            const uint16_t *ab = ad_b + (size_t)next * m * ad.rank;
            for (int i = 0; i < TM; ++i) {
                int mr = m0 + 16 * i + r;
                mr = mr < m ? mr : m - 1;
                f32x4 p[TN];
#pragma unroll
                for (int j = 0; j < TN; ++j) p[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                for (int kk = 0; kk < ad.rank_pad; kk += 32) {
                    uint16_t q[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        q[c] = kk + 8 * g + c < ad.rank
                                   ? ab[(size_t)mr * ad.rank + kk + 8 * g + c] : (uint16_t)0;
                    u32x4 a;
#pragma unroll
                    for (int c = 0; c < 4; ++c) a[c] = q[2 * c] | ((uint32_t)q[2 * c + 1] << 16);
#pragma unroll
                    for (int j = 0; j < TN; ++j) {
                        int64_t tok = t0 + 16 * j + r;
                        tok = tok < hi ? tok : hi - 1;
                        const u32x4 b = *reinterpret_cast<const u32x4 *>(v + tok * ad.rank_pad + kk + 8 * g);
                        p[j] = Act<BF>::mfma(a, b, p[j]);
                    }
                }
#pragma unroll
                for (int ii = 0; ii < TM; ++ii)
                    if (ii == i)
#pragma unroll
                        for (int j = 0; j < TN; ++j)
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                acc[ii][j][c] += idj[j] == next ? p[j][c] : 0.0f;
            }
        }
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        const int64_t tok = t0 + 16 * j + r;
        if (tok >= hi) continue;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int col = m0 + 16 * i + 4 * g;
            if (col >= m) continue;
            uint16_t *o = y + tok * ldy + col;
#pragma unroll
            for (int c = 0; c < 4; ++c) o[c] = Act<BF>::store(acc[i][j][c]);
        }
    }
}

__global__ void __launch_bounds__(256)
pack_rows_kernel(const uint16_t *__restrict__ x, int64_t ldx, int64_t n, int k,
                 uint16_t *__restrict__ out) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n * (k / 8)) return;
    const int64_t row = i / (k / 8);
    const int c = (int)(i - row * (k / 8)) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) out[row * k + c + j] = x[row * ldx + c + j];
}

__global__ void __launch_bounds__(256)
zero_rows_kernel(const int32_t *__restrict__ offsets, int groups, int64_t n, int m,
                 uint16_t *__restrict__ y, int64_t ldy) {
    const int64_t row = blockIdx.x;
    if (row >= offsets[0] && row < offsets[groups]) return;
    for (int c = threadIdx.x; c < m; c += 256) y[row * ldy + c] = 0;
}

template <int LV, int K, int HB>
hipError_t dense_t(const WeightArgs &w, const int32_t *offsets, int64_t n, int g0, int ng,
                   bool transposed, bool bf16, uint16_t *dense, hipStream_t stream) {
    const dim3 grid((unsigned)(w.rows / HB * (w.cols / HB)), (unsigned)ng);
#define EXL3_DENSE(BF, TR)                                                                     \
    hipLaunchKernelGGL((dense_kernel<LV, K, HB, BF, TR>), grid, dim3(HB * 4), 0, stream,       \
                       w.packed, w.lv, w.rows, w.cols, w.K, w.scale, w.su, w.sv, offsets, n, g0, \
                       dense)
    if (bf16 && transposed)
        EXL3_DENSE(true, true);
    else if (bf16)
        EXL3_DENSE(true, false);
    else if (transposed)
        EXL3_DENSE(false, true);
    else
        EXL3_DENSE(false, false);
#undef EXL3_DENSE
    return hipGetLastError();
}

template <int LV, int K>
hipError_t dense_h(const WeightArgs &w, const int32_t *offsets, int64_t n, int g0, int ng,
                   bool transposed, bool bf16, uint16_t *dense, hipStream_t stream) {
    return w.had == 128
               ? dense_t<LV, K, 128>(w, offsets, n, g0, ng, transposed, bf16, dense, stream)
               : dense_t<LV, K, 64>(w, offsets, n, g0, ng, transposed, bf16, dense, stream);
}

}  // namespace

hipError_t launch_dense(const WeightArgs &w, const int32_t *offsets, int64_t n, int g0, int ng,
                        bool transposed, bool bf16, uint16_t *dense, hipStream_t stream) {
#define EXL3_DENSE_K(LV, KK) \
    case KK: return dense_h<LV, KK>(w, offsets, n, g0, ng, transposed, bf16, dense, stream)
    if (w.lv_kind == kLevelsMul1)
        switch (w.K) {
            EXL3_DENSE_K(kLevelsMul1, 1);
            EXL3_DENSE_K(kLevelsMul1, 2);
            EXL3_DENSE_K(kLevelsMul1, 3);
            EXL3_DENSE_K(kLevelsMul1, 4);
        }
    else if (w.lv_kind == kLevelsHalves)
        switch (w.K) {
            EXL3_DENSE_K(kLevelsHalves, 1);
            EXL3_DENSE_K(kLevelsHalves, 2);
            EXL3_DENSE_K(kLevelsHalves, 3);
            EXL3_DENSE_K(kLevelsHalves, 4);
        }
#undef EXL3_DENSE_K
    return dense_h<kLevelsTable, 0>(w, offsets, n, g0, ng, transposed, bf16, dense, stream);
}

hipError_t launch_gemm(const void *x, int64_t ldx, const uint16_t *dense, int64_t n, int m, int k,
                       const int32_t *offsets, int g0, int ng, bool bf16,
                       const AdapterArgs *ad, const void *b, const uint16_t *v, void *y,
                       int64_t ldy, int n_cu, hipStream_t stream) {
    const AdapterArgs args = ad ? *ad : AdapterArgs{};
    const uint16_t *xx = static_cast<const uint16_t *>(x), *bb = static_cast<const uint16_t *>(b);
    uint16_t *yy = static_cast<uint16_t *>(y);
#define EXL3_GEMM(BM, BN, WM, WN, BF)                                                            \
    do {                                                                                         \
        const int m_tiles = (m + BM - 1) / BM;                                                   \
        const int64_t n_tiles = offsets ? n / BN + ng : (n + BN - 1) / BN;                       \
        const int total = (int)(m_tiles * n_tiles);                                              \
        hipLaunchKernelGGL((gemm_kernel<BM, BN, WM, WN, BF>), dim3((unsigned)total),             \
                           dim3(64 * WM * WN), 0, stream, xx, ldx, dense, n, m, k, offsets, g0,  \
                           ng, m_tiles, total, args, bb, v, yy, ldy);                            \
    } while (0)
    // the large tile needs a workgroup for most compute units to be worth it
    const int64_t large = (int64_t)((m + 255) / 256) * ((n + 255) / 256);
    if (!offsets && large >= n_cu / 2) {
        if (bf16)
            EXL3_GEMM(256, 256, 2, 4, true);
        else
            EXL3_GEMM(256, 256, 2, 4, false);
    } else {
        if (bf16)
            EXL3_GEMM(128, 128, 2, 2, true);
        else
            EXL3_GEMM(128, 128, 2, 2, false);
    }
#undef EXL3_GEMM
    return hipGetLastError();
}

hipError_t launch_pack_rows(const void *x, int64_t ldx, int64_t n, int k, uint16_t *out,
                            hipStream_t stream) {
    const unsigned grid = (unsigned)((n * (k / 8) + 255) / 256);
    hipLaunchKernelGGL(pack_rows_kernel, dim3(grid), dim3(256), 0, stream,
                       static_cast<const uint16_t *>(x), ldx, n, k, out);
    return hipGetLastError();
}

hipError_t launch_zero_rows(const int32_t *offsets, int groups, int64_t n, int m, void *y,
                            int64_t ldy, hipStream_t stream) {
    hipLaunchKernelGGL(zero_rows_kernel, dim3((unsigned)n), dim3(256), 0, stream, offsets, groups,
                       n, m, static_cast<uint16_t *>(y), ldy);
    return hipGetLastError();
}

}  // namespace exl3
