// Products of many rows with coded weights on gfx950: the weights written once
// in the activations' type and their own domain (dense_kernel), then a matrix
// product (gemm_kernel).  Both directions, y = x W^T and y = x W, contract over
// consecutive elements: for the second the weights are written transposed.
#include "coded.h"

namespace exl3 {

namespace {

__device__ __forceinline__ uint32_t parity16(uint32_t v) { return __popc(v) & 1u; }

// ---- dense weights ----
// A workgroup takes an HB x HB block of W (HB: the Hadamard block), a wave per
// 16 rows and then per 16 columns.  Both transforms run
// on the matrix units: the levels are exact in binary16 and the transform's
// entries are +-1, held as operands made once.
//   1. The wave decodes 16 x 64 levels into operands (coded.h) and multiplies
//      them by H_64 over their columns: entry (c, n) is (-1)^popcount(c & n).
//      For HB = 128 the halves' sum and difference follow.
//   2. The result, sums of HB levels, passes through shared memory column by
//      column as binary16: for bfloat16 weights rounded to it (at most 2^-11 of each,
//      an eighth of what the final rounding takes), for binary16 weights in two
//      parts, the rounded value and the rest, so that the weights are rounded
//      once.  The codebooks' levels are below 4 and their sums below 2^9; a
//      caller's table may hold any binary16 value, and its sums take the power of
//      two that brings its largest level there (Levels::norm, exact both ways).
//   3. The wave transforms 16 columns over the rows.  Of a row's index in H_HB
//      the lowest five bits meet the matrix instruction's 32 k's; the sums over
//      the remaining index are butterflies of the results.
// Then the scale, su and sv in binary32 and one rounding to the activations'
// type.  Binary16 has too few exponents for any su and sv: its weights are stored
// without the powers of two of their scale and of their result's channel, and
// divided by that of the largest factor on the contracted side, below 2^15 and,
// where the levels are spread evenly, some 2^4; the product's results get them back
// (gemm_kernel).  What is below 2^-18 of a channel's spread alone is rounded to
// fewer bits.  Row-major and transposed output differ in the order of step 3's
// operands: either way a lane holds four consecutive elements of the output.
// 4096 x 4096, K = 2: 13.3 to 15 us, 2.5 TB/s written; the chain of decoding,
// products and two passes through shared memory in each workgroup bounds it more
// than the write (7.1 us) does.
template <int LV, int K, int HB, bool BF, bool TR>
__global__ void __launch_bounds__(HB * 4, 4)
dense_kernel(const uint32_t *__restrict__ packed, Levels lv, int rows, int cols, int Kr,
             const float *__restrict__ scale, const float *__restrict__ su,
             const float *__restrict__ sv, const int32_t *__restrict__ offsets, int64_t n, int g0,
             const int32_t *__restrict__ inner, uint16_t *__restrict__ dense,
             uint16_t *__restrict__ y, int64_t ldy, int groups) {
    constexpr int kPitch = HB * 2 + 16;          // bytes a column of the block takes in LDS
    constexpr int kParts = BF ? 1 : 2, NT = HB / 16, NP = HB / 32;
    __shared__ __align__(16) char mid[kParts][HB * kPitch];
    const int lane = threadIdx.x & 63, wv = wave_number();
    const int r = lane & 15, g = lane >> 4;
    const int e = g0 + blockIdx.y, blocks = cols / HB;
    const int br = blockIdx.x / blocks, bc = blockIdx.x % blocks;
    int64_t lo, hi;
    if (offsets && g0 == 0) {
        // rows of y before the first group and after the last, by all workgroups
        const int64_t from = offsets[0], to = offsets[groups];
        const int64_t all = (int64_t)gridDim.x * gridDim.y;
        const int64_t me = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
        const int m = TR ? cols : rows;
        for (int64_t t = me; t < n && t < from; t += all)
            for (int c = threadIdx.x; c < m; c += HB * 4) y[t * ldy + c] = 0;
        for (int64_t t = (to > 0 ? to : 0) + me; t < n; t += all)
            for (int c = threadIdx.x; c < m; c += HB * 4) y[t * ldy + c] = 0;
    }
    group_rows(offsets, e, n, lo, hi);
    if (lo >= hi) return;                        // no row uses this group
    const int kk = K ? K : Kr;
    const uint32_t *tiles = packed + (((size_t)e * (rows / 16) + br * NT + wv) * (cols / 16) + g) *
                                         (8 * kk);
    // the words come first, the operands of signs are made meanwhile
    uint32_t d[HB / 64][RowWords<K>::N];
#pragma unroll
    for (int q = 0; q < HB / 64; ++q)
        load_row<K>(tiles + (size_t)(bc * NT + 4 * q) * (8 * kk), r, d[q]);
    // operands of signs: column (or row) r against k's low four bits 8 s + j
    u32x4 low[2];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            low[s][j] = 0x3C003C00u | (parity16((8 * s + 2 * j) & r) << 15) |
                        (parity16((8 * s + 2 * j + 1) & r) << 31);
    u32x4 h64[4][2];                             // H_64 at k = 16 g + 8 s + j, column 16 t + r
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const uint32_t flip = parity16(g & t) ? 0x80008000u : 0u;
#pragma unroll
        for (int s = 0; s < 2; ++s) h64[t][s] = low[s] ^ flip;
    }
    // H_32 at row 16 o + r, k = 8 g + j
    u32x4 h32[2];
    h32[0] = (g & 1) ? low[1] : low[0];
    h32[1] = h32[0] ^ ((g >> 1) ? 0x80008000u : 0u);
    const float norm = LV == kLevelsTable ? lv.norm : 1.0f;
    float f = scale[e] / ((float)HB * norm);
    int down = 0;                                // powers of two taken off the contracted side
    if (!BF) {
        f = __builtin_amdgcn_frexp_mantf(f);
        down = -(inner[e] + 1);
    }
    // the factors of the result's side, and of the contracted one
    auto outer_factor = [&](float s) { return f * (BF ? s : __builtin_amdgcn_frexp_mantf(s)); };
    auto inner_factor = [&](float s) { return BF ? s : __builtin_ldexpf(s, down); };
    const float *su_b = su + (size_t)e * rows + (size_t)br * HB;
    float su_t[TR ? 1 : NT];
    if (!TR)
#pragma unroll
        for (int t = 0; t < NT; ++t) su_t[t] = outer_factor(su_b[16 * t + r]);
    uint16_t *out = dense + (size_t)blockIdx.y * rows * cols;

    f32x4 sum[NT];
#pragma unroll
    for (int q = 0; q < HB / 64; ++q) {
        u32x4 w[2];
        decode_row<LV, K>(tiles + (size_t)(bc * NT + 4 * q) * (8 * kk), r, d[q], lv, w);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            f32x4 p = {0.0f, 0.0f, 0.0f, 0.0f};
            p = Act<false>::mfma(w[0], h64[t][0], p);
            p = Act<false>::mfma(w[1], h64[t][1], p);
            if (q == 0) {
                sum[t] = p;
            } else {
                sum[(4 + t) % NT] = sum[t] - p;
                sum[t] = sum[t] + p;
            }
        }
    }
    // column 16 t + r, rows 16 wv + 4 g .. + 3
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        if (LV == kLevelsTable) sum[t] *= norm;
        f16x2 a, b;
        a[0] = (_Float16)sum[t][0];
        a[1] = (_Float16)sum[t][1];
        b[0] = (_Float16)sum[t][2];
        b[1] = (_Float16)sum[t][3];
        const int at = (16 * t + r) * kPitch + (16 * wv + 4 * g) * 2;
        *reinterpret_cast<uint2 *>(mid[0] + at) =
            uint2{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
        if (!BF) {
            f16x2 c, dd;
            c[0] = (_Float16)(sum[t][0] - (float)a[0]);
            c[1] = (_Float16)(sum[t][1] - (float)a[1]);
            dd[0] = (_Float16)(sum[t][2] - (float)b[0]);
            dd[1] = (_Float16)(sum[t][3] - (float)b[1]);
            *reinterpret_cast<uint2 *>(mid[kParts - 1] + at) =
                uint2{__builtin_bit_cast(uint32_t, c), __builtin_bit_cast(uint32_t, dd)};
        }
    }
    __syncthreads();
    // sums over 32 rows p for the two values of the row index's fifth bit,
    // then over the p's
    f32x4 z[NT];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int at = (16 * wv + r) * kPitch + (32 * p + 8 * g) * 2;
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            f32x4 a = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int q = 0; q < kParts; ++q) {
                const u32x4 m = *reinterpret_cast<const u32x4 *>(mid[q] + at);
                a = TR ? Act<false>::mfma(h32[o], m, a) : Act<false>::mfma(m, h32[o], a);
            }
            z[2 * p + o] = a;
        }
    }
#pragma unroll
    for (int s = 2; s < NT; s <<= 1)
#pragma unroll
        for (int t = 0; t < NT; ++t)
            if (!(t & s)) {
                const f32x4 a = z[t], b = z[t + s];
                z[t] = a + b;
                z[t + s] = a - b;
            }
    // transposed: column 16 wv + r, rows 16 t + 4 g ..; else row 16 t + r,
    // columns 16 wv + 4 g ..
    const float *sv_b = sv + (size_t)e * cols + (size_t)bc * HB + 16 * wv;
    float sv_r = 0.0f;
    f32x4 sv_4 = {0.0f, 0.0f, 0.0f, 0.0f};
    if (TR)
        sv_r = outer_factor(sv_b[r]);
    else
        sv_4 = *reinterpret_cast<const f32x4u *>(sv_b + 4 * g);
    __syncthreads();                         // the halves have been read
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        f32x4 v = z[t];
        if (TR) {
            const f32x4 s4 = *reinterpret_cast<const f32x4u *>(su_b + 16 * t + 4 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] *= sv_r * inner_factor(s4[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] *= su_t[t] * inner_factor(sv_4[i]);
        }
        char *at = TR ? mid[0] + (16 * wv + r) * kPitch + (16 * t + 4 * g) * 2
                      : mid[0] + (16 * t + r) * kPitch + (16 * wv + 4 * g) * 2;
        *reinterpret_cast<uint2 *>(at) =
            uint2{Act<BF>::store2(v[0], v[1]), Act<BF>::store2(v[2], v[3])};
    }
    __syncthreads();
    // whole rows of the block to memory
    const size_t pitch = TR ? rows : cols;
    uint16_t *o0 = out + (TR ? (size_t)bc : (size_t)br) * HB * pitch +
                   (TR ? (size_t)br : (size_t)bc) * HB;
#pragma unroll
    for (int i = 0; i < HB / 32; ++i) {
        const int piece = i * HB * 4 + threadIdx.x, row = piece / (HB / 8);
        const int c = piece % (HB / 8);
        *reinterpret_cast<u32x4 *>(o0 + row * pitch + c * 8) =
            *reinterpret_cast<const u32x4 *>(mid[0] + row * kPitch + c * 16);
    }
}

// The exponent of the largest of each group's k factors (a workgroup a group).
// Latency bounds it: 3 us for 4,096 factors; found in every workgroup of
// dense_kernel instead, beside its other loads, it lengthened that by as much.
__global__ void __launch_bounds__(512)
inner_kernel(const float *__restrict__ factors, int k, int32_t *__restrict__ inner) {
    __shared__ uint32_t wave_big[8];
    const float *at = factors + (size_t)blockIdx.x * k;
    uint32_t big = 0;                            // magnitudes compare as integers
    for (int c = threadIdx.x * 4; c < k; c += 2048) {
        const f32x4 v = *reinterpret_cast<const f32x4u *>(at + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float one = v[i];              // (of a vector's element itself a bit cast is
                                                 // that of the first)
            const uint32_t m = __builtin_bit_cast(uint32_t, one) & 0x7FFFFFFFu;
            big = m > big ? m : big;
        }
    }
    for (int m = 1; m < 64; m <<= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)big, m);
        big = o > big ? o : big;
    }
    if ((threadIdx.x & 63) == 0) wave_big[threadIdx.x >> 6] = big;
    __syncthreads();
    if (threadIdx.x) return;
    for (int i = 1; i < 8; ++i) big = wave_big[i] > big ? wave_big[i] : big;
    inner[blockIdx.x] = __builtin_amdgcn_frexp_expf(__builtin_bit_cast(float, big));
}

// ---- matrix product ----
// y[n][m] = x[n][k] w[m][k]^T: the weights are the instruction's first operand
// and the rows of x its second, so a lane's four results are consecutive
// elements of one row of y.  A workgroup computes BM columns of y by BN rows.
// Slices of 64 k (whole cache lines) pass through two places in shared memory,
// loaded straight into them.  While the matrix units work on one half slice the
// next one's operands are read into registers: those of x beside the present
// ones, those of the weights over them, row by row as they are used up.  The one
// barrier a slice stands where its second half has just been read: the slice's
// place is free for the slice after the next, whose loads get the time of a whole
// slice to land.  A load writes a wave's 64 pieces of 16 bytes in lane order, so
// the swizzle that spreads rows over the banks is in which piece each lane
// fetches: piece s of row r holds k piece s ^ (r & 7), whose reads meet no bank
// twice (4.2 cycles a read of 1 KiB measured, where a swizzle by three other
// bits of r took 8.1).  4,096 rows, 12288 x 4096, bfloat16: 300 us, 1,375 TFLOP/s,
// its matrix units busy for 72 % of the cycles; the rest is mostly the barrier and
// the reads it waits for, once a slice.
template <int BM, int BN, int WM, int WN, bool BF, bool AD>
__global__ void __launch_bounds__(64 * WM * WN, 2)
gemm_kernel(const uint16_t *__restrict__ x, int64_t ldx, const uint16_t *__restrict__ w,
            DenseScale ds, int64_t n, int m, int k, const int32_t *__restrict__ offsets, int g0, int ng, int m_tiles,
            int total, AdapterArgs ad, const uint16_t *__restrict__ ad_b,
            const uint16_t *__restrict__ v, uint16_t *__restrict__ y, int64_t ldy) {
    constexpr int kThreads = 64 * WM * WN, SM = BM / WM, SN = BN / WN, TM = SM / 16, TN = SN / 16;
    constexpr int kPiecesW = BM * 8 / kThreads, kPiecesX = BN * 8 / kThreads;
    constexpr int kPieces = kPiecesW + kPiecesX;          // 16-byte pieces a thread loads a slice
    constexpr int kSlice = (BM + BN) * 64, kRing = 2;
    constexpr int kPitch = SM * 2 + 16;                   // bytes a row of y takes in the epilogue
    static_assert(WM * WN * 16 * kPitch <= kRing * kSlice * 2, "the epilogue fits the ring");
    __shared__ __align__(16) uint16_t ring[kRing * kSlice];
    const int lane = threadIdx.x & 63, wv = wave_number();
    const int r = lane & 15, g = lane >> 4, wm = wv % WM, wn = wv / WM;
    // each die takes a run of tiles
    if (offsets) {
        total = count_tiles(offsets, g0, ng, n, BN, total / m_tiles) * m_tiles;
        if ((int)blockIdx.x >= total) return;    // fewer tiles than the grid allows for
    }
    int id = tile_of_die(blockIdx.x, total);
    // and orders them in panels eight tiles wide, so that the 32 tiles a
    // die works on at a time share their operands in its cache in both
    // directions (one row of 32 tiles fetches 2.75 times what 8 x 4 do)
    const int n_tiles = total / m_tiles, panel = id / (8 * n_tiles);
    const int wide = m_tiles - 8 * panel < 8 ? m_tiles - 8 * panel : 8;
    id -= 8 * panel * n_tiles;
    const int mt = 8 * panel + id % wide;
    int nt = id / wide, e = 0;
    int64_t lo = 0, hi = n;
    if (offsets) {
        e = group_of_tile(offsets, g0, ng, n, BN, nt);
        if (e < 0) return;
        group_rows(offsets, e, n, lo, hi);
        e -= g0;
    }
    const int64_t row0 = lo + (int64_t)nt * BN;
    // the tile's operands from uniform bases that move along k, and 32-bit
    // offsets of the thread's pieces
    const char *w_at = reinterpret_cast<const char *>(w + ((size_t)e * m + (size_t)mt * BM) * k);
    const char *x_at = reinterpret_cast<const char *>(x + row0 * ldx);
    uint32_t piece_at[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const int q = (i < kPiecesW ? i : i - kPiecesW) * kThreads + threadIdx.x, row = q >> 3;
        const int kp = ((q & 7) ^ (row & 7)) * 16;
        if (i < kPiecesW) {
            const int left = m - mt * BM - 1;    // past the edge: repeats, not stored
            piece_at[i] = (uint32_t)(row < left ? row : left) * (uint32_t)(k * 2) + kp;
        } else {
            const int64_t left = hi - row0 - 1;
            piece_at[i] = (uint32_t)(row < left ? row : left) * (uint32_t)(ldx * 2) + kp;
        }
    }
    const int steps = k / 64;
    auto load_piece = [&](int i, int place) {
        const int q = i < kPiecesW ? i : BM * 8 / kThreads + i - kPiecesW;
        load_to_lds((i < kPiecesW ? w_at : x_at) + piece_at[i],
                    ring + place * kSlice + (q * kThreads + wv * 64) * 8);
    };
    // to the next slice; the last is repeated into the place that nobody reads
    auto advance = [&](int loaded) {
        const int by = loaded < steps ? 128 : 0;
        w_at += by;
        x_at += by;
    };
    u32x4 a[TM], b[2][TN];
    const int at[2] = {(g ^ (r & 7)) * 8, ((4 + g) ^ (r & 7)) * 8};
    const uint16_t *ra = ring + (wm * SM + r) * 64, *rb = ring + (BM + wn * SN + r) * 64;
    auto read_a = [&](int i, int place, int half) {
        a[i] = *reinterpret_cast<const u32x4 *>(ra + place * kSlice + 16 * i * 64 + at[half]);
    };
    auto read_b = [&](int j, int place, int half) {
        b[half][j] = *reinterpret_cast<const u32x4 *>(rb + place * kSlice + 16 * j * 64 + at[half]);
    };
    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kPieces; ++i) load_piece(i, 0);
    advance(1);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) load_piece(i, 1);
    advance(2);
    wait_loads<kPieces>();
    barrier_in_place();
#pragma unroll
    for (int j = 0; j < TN; ++j) read_b(j, 0, 0);
#pragma unroll
    for (int i = 0; i < TM; ++i) read_a(i, 0, 0);
    auto products = [&](int i, int half) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = Act<BF>::mfma(a[i], b[half][j], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
    };
    for (int s = 0; s < steps; ++s) {
        const int place = s & 1;
        // the first half; the second is read
#pragma unroll
        for (int i = 0; i < TM; ++i) {
#pragma unroll
            for (int j = i * TN / TM; j < (i + 1) * TN / TM; ++j) read_b(j, place, 1);
            products(i, 0);
            read_a(i, place, 1);
        }
        // the second half; the next slice's first is read, the one after loaded
        products(0, 1);
        wait_loads<0>();
        barrier_in_place();
        read_a(0, place ^ 1, 0);
#pragma unroll
        for (int i = 1; i < TM; ++i) {
#pragma unroll
            for (int j = (i - 1) * TN / (TM - 1); j < i * TN / (TM - 1); ++j)
                read_b(j, place ^ 1, 0);
#pragma unroll
            for (int q = (i - 1) * kPieces / (TM - 1); q < i * kPieces / (TM - 1); ++q)
                load_piece(q, place);
            products(i, 1);
            read_a(i, place ^ 1, 0);
        }
        advance(s + 3);
    }
    const int m0 = mt * BM + wm * SM;
    const int64_t t0 = row0 + wn * SN;
    if (!BF) {
        // the powers of two that the weights were divided by
        const int eg = g0 + e;
        const int all = __builtin_amdgcn_frexp_expf(ds.scale[eg] / ds.div) + ds.inner[eg] + 1;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int mr = m0 + 16 * i + 4 * g;  // past the edge: repeats, not stored
            const f32x4 s = *reinterpret_cast<const f32x4u *>(ds.out + (size_t)eg * m +
                                                              (mr < m ? mr : m - 4));
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int up = all + __builtin_amdgcn_frexp_expf(s[c]);
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j][c] = __builtin_ldexpf(acc[i][j][c], up);
            }
        }
    }
    if (AD) {
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
            const uint16_t *end = ad_b + (size_t)ad.count * m * ad.rank;
            for (int kk = 0; kk < ad.rank_pad; kk += 32) {
                // operands ahead of their products, the weights' side made zero past
                // the rank
                const int valid = ad.rank - kk - 8 * g;
                u32x4 keep, av[TM], bv[TN];
                float vs[TN];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    keep[c] = valid >= 2 * c + 2 ? 0xFFFFFFFFu : valid == 2 * c + 1 ? 0xFFFFu : 0u;
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    int mr = m0 + 16 * i + r;
                    mr = mr < m ? mr : m - 1;
                    const uint16_t *ap = ab + (size_t)mr * ad.rank + kk + 8 * g;
                    av[i] = u32x4{0u, 0u, 0u, 0u};
                    if (valid > 0) {
                        if (end - ap >= 8)
                            av[i] = *reinterpret_cast<const u32x4u *>(ap);
                        else
                            for (int c = 0; c < valid; ++c)
                                av[i][c >> 1] |= (uint32_t)ap[c] << (16 * (c & 1));
                    }
                }
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    int64_t tok = t0 + 16 * j + r;
                    tok = tok < hi ? tok : hi - 1;
                    bv[j] = *reinterpret_cast<const u32x4 *>(v + tok * ad.rank_pad + kk + 8 * g);
                    vs[j] = BF ? 1.0f : ad.vs[tok];
                }
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j) {
                        f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
                        z = Act<BF>::mfma(av[i] & keep, bv[j], z);
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            acc[i][j][c] += idj[j] == next ? (BF ? z[c] : z[c] * vs[j]) : 0.0f;
                    }
            }
        }
    }
    // 16 rows of y at a time through the wave's part of the ring, so that whole
    // lines are written
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    char *out = reinterpret_cast<char *>(ring) + wv * 16 * kPitch;
    constexpr int kPer = SM / 8;             // 16-byte pieces a row
#pragma unroll
    for (int j = 0; j < TN; ++j) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
            *reinterpret_cast<uint2 *>(out + r * kPitch + (16 * i + 4 * g) * 2) =
                uint2{Act<BF>::store2(acc[i][j][0], acc[i][j][1]),
                      Act<BF>::store2(acc[i][j][2], acc[i][j][3])};
#pragma unroll
        for (int q = 0; q < 16 * kPer / 64; ++q) {
            const int piece = q * 64 + lane, row = piece / kPer, c = piece % kPer * 8;
            const u32x4 o = *reinterpret_cast<const u32x4 *>(out + row * kPitch + c * 2);
            const int64_t tok = t0 + 16 * j + row;
            if (tok >= hi || m0 + c >= m) continue;
            uint16_t *yo = y + tok * ldy + m0 + c;
            *reinterpret_cast<u32x4u *>(yo) = o;
        }
    }
}

__global__ void __launch_bounds__(256)
pack_rows_kernel(const uint16_t *__restrict__ x, int64_t ldx, int64_t n, int k,
                 uint16_t *__restrict__ out) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n * (k / 8)) return;                // the rows of one launch
    const int64_t row = i / (k / 8);
    const int c = (int)(i - row * (k / 8)) * 8;
    *reinterpret_cast<u32x4 *>(out + row * k + c) =
        *reinterpret_cast<const u32x4u *>(x + row * ldx + c);
}

template <int LV, int K, int HB>
hipError_t dense_t(const WeightArgs &w, const int32_t *offsets, int64_t n, int g0, int ng,
                   bool transposed, bool bf16, const int32_t *inner, uint16_t *dense,
                   uint16_t *y, int64_t ldy, hipStream_t stream) {
    const dim3 grid((unsigned)(w.rows / HB * (w.cols / HB)), (unsigned)ng);
#define EXL3_DENSE(BF, TR)                                                                     \
    hipLaunchKernelGGL((dense_kernel<LV, K, HB, BF, TR>), grid, dim3(HB * 4), 0, stream,       \
                       w.packed, w.lv, w.rows, w.cols, w.K, w.scale, w.su, w.sv, offsets, n, g0, \
                       inner, dense, y, ldy, w.groups)
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
                   bool transposed, bool bf16, const int32_t *inner, uint16_t *dense,
                   uint16_t *y, int64_t ldy, hipStream_t stream) {
    return w.had == 128 ? dense_t<LV, K, 128>(w, offsets, n, g0, ng, transposed, bf16, inner, dense,
                                              y, ldy, stream)
                        : dense_t<LV, K, 64>(w, offsets, n, g0, ng, transposed, bf16, inner, dense,
                                             y, ldy, stream);
}

}  // namespace

hipError_t launch_dense(const WeightArgs &w, const int32_t *offsets, int64_t n, int g0, int ng,
                        bool transposed, bool bf16, const int32_t *inner, uint16_t *dense, void *yv,
                        int64_t ldy, hipStream_t stream) {
    uint16_t *y = static_cast<uint16_t *>(yv);
#define EXL3_DENSE_K(LV, KK) \
    case KK:                     \
        return dense_h<LV, KK>(w, offsets, n, g0, ng, transposed, bf16, inner, dense, y, ldy, stream)
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
    return dense_h<kLevelsTable, 0>(w, offsets, n, g0, ng, transposed, bf16, inner, dense, y, ldy,
                                    stream);
}

hipError_t launch_inner(const WeightArgs &w, bool transposed, int32_t *inner, hipStream_t stream) {
    hipLaunchKernelGGL(inner_kernel, dim3((unsigned)w.groups), dim3(512), 0, stream,
                       transposed ? w.su : w.sv, transposed ? w.rows : w.cols, inner);
    return hipGetLastError();
}

hipError_t launch_gemm(const void *x, int64_t ldx, const uint16_t *dense, const DenseScale &ds,
                       int64_t n, int m, int k, const int32_t *offsets, int g0, int ng, bool bf16,
                       const AdapterArgs *ad, const void *b, const uint16_t *v, void *y,
                       int64_t ldy, int n_cu, hipStream_t stream) {
    const AdapterArgs args = ad ? *ad : AdapterArgs{};
    const uint16_t *xx = static_cast<const uint16_t *>(x), *bb = static_cast<const uint16_t *>(b);
    uint16_t *yy = static_cast<uint16_t *>(y);
#define EXL3_GEMM_T(BM, BN, WM, WN, BF, AD)                                                      \
    hipLaunchKernelGGL((gemm_kernel<BM, BN, WM, WN, BF, AD>), dim3((unsigned)total),             \
                       dim3(64 * WM * WN), 0, stream, xx, ldx, dense, ds, n, m, k, offsets, g0,  \
                       ng, m_tiles, total, args, bb, v, yy, ldy)
#define EXL3_GEMM(BM, BN, WM, WN)                                                                \
    do {                                                                                         \
        const int m_tiles = (m + BM - 1) / BM;                                                   \
        const int64_t n_tiles = offsets ? n / BN + ng : (n + BN - 1) / BN;                       \
        const int total = (int)(m_tiles * n_tiles);                                              \
        if (bf16 && ad)                                                                          \
            EXL3_GEMM_T(BM, BN, WM, WN, true, true);                                             \
        else if (bf16)                                                                           \
            EXL3_GEMM_T(BM, BN, WM, WN, true, false);                                            \
        else if (ad)                                                                             \
            EXL3_GEMM_T(BM, BN, WM, WN, false, true);                                            \
        else                                                                                     \
            EXL3_GEMM_T(BM, BN, WM, WN, false, false);                                           \
    } while (0)
    // What a round of tiles takes at k = 4096, us: one tile a compute unit, of the
    // smallest two (40 for half a round of these); a group's last tile counts as
    // whole.  1,500 rows x 4,096 columns: 56 in 256 tiles of 128 x 192, 64 in 192 of
    // 128 x 256; 5,000 rows: 149 in two rounds of 256 x 192, 194 in two of 256 x 256.
    auto tiles = [&](int bm, int bn) {
        return (int64_t)((m + bm - 1) / bm) * (offsets ? n / bn + ng : (n + bn - 1) / bn);
    };
    auto rounds = [&](int64_t t) { return (t + n_cu - 1) / n_cu; };
    const int64_t small = tiles(128, 128), rest = small % (2 * n_cu);
    const int64_t cost[5] = {97 * rounds(tiles(256, 256)), 82 * rounds(tiles(256, 192)),
                             62 * rounds(tiles(128, 256)), 54 * rounds(tiles(128, 192)),
                             65 * (small / (2 * n_cu)) +
                                 (rest > n_cu ? 65 : rest > 0 ? 40 : 0)};
    int best = 0;
    for (int i = 1; i < 5; ++i)
        if (cost[i] < cost[best]) best = i;
    switch (best) {
        case 0: EXL3_GEMM(256, 256, 2, 4); break;
        case 1: EXL3_GEMM(256, 192, 2, 4); break;
        case 2: EXL3_GEMM(128, 256, 2, 4); break;
        case 3: EXL3_GEMM(128, 192, 2, 4); break;
        default: EXL3_GEMM(128, 128, 2, 2);
    }
#undef EXL3_GEMM_T
#undef EXL3_GEMM
    return hipGetLastError();
}

hipError_t launch_pack_rows(const void *x, int64_t ldx, int64_t n, int k, uint16_t *out,
                            hipStream_t stream) {
    const int64_t per = rows_a_launch(k / 8);
    for (int64_t r0 = 0; r0 < n; r0 += per) {
        const int64_t rows = n - r0 < per ? n - r0 : per;
        const unsigned grid = (unsigned)((rows * (k / 8) + 255) / 256);
        hipLaunchKernelGGL(pack_rows_kernel, dim3(grid), dim3(256), 0, stream,
                           static_cast<const uint16_t *>(x) + r0 * ldx, ldx, rows, k, out + r0 * k);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace exl3
