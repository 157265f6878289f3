// Matrix products in 8-bit blocks (gfx950): y = x W^T and x W with codes in e4m3 and a scale for
// each block of 128 along the contraction.
//
//   y[t][m] = sum over blocks b of sx[t][b] sw[m / 128][b] (sum over k in b of x[t][k] w[m][k])
//
// One matrix instruction, 16 x 16 x 128, contracts exactly one block: its result is scaled and
// added to the running sums in binary32.  The weights are its first operand and the rows of x its
// second, so a lane's four results belong to one row of x and to one 128-row block of W, and one
// factor serves all four.  Which k's a lane holds is free as long as both operands agree: lane
// group g = lane >> 4 takes the 16-byte pieces g and 4 + g of a block's 128 bytes.
#include "blocks.h"

namespace exl3 {

namespace {

using i32x8 = int __attribute__((ext_vector_type(8)));

struct Operand {
    u32x4 a, b;                                  // pieces g and 4 + g
};
__device__ __forceinline__ f32x4 block_product(const Operand &w, const Operand &x) {
    i32x8 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[i] = (int)w.a[i];
        a[4 + i] = (int)w.b[i];
        b[i] = (int)x.a[i];
        b[4 + i] = (int)x.b[i];
    }
    // both formats e4m3, scales of one
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0,
                                                            0, 0, 0, 0, 0);
}

// Turns 8 x 16 bytes: of 16 lanes, lane 2 j + q names bytes 8 q .. 8 q + 7 of row j, and lane i
// gets byte i of rows 0..7.
using i32x2 = int __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u32x2 read_turned8(const uint8_t *from) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32(
        (__attribute__((address_space(3))) i32x2 *)from));
}

// Four bytes a lane straight into shared memory, at to + 4 lane.
__device__ __forceinline__ void load4_to_lds(const void *from, void *to) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from,
                                     (__attribute__((address_space(3))) void *)to, 4, 0, 0);
}

// Sets the rows of y before the first group and from the last offset on to zero; all workgroups
// of the grid take part.
__device__ __forceinline__ void clear_rows_of_no_group(const int32_t *offsets, int groups,
                                                       int64_t n, uint16_t *y, int64_t ldy, int m) {
    const int64_t from = offsets[0], to = offsets[groups];
    const int64_t all = gridDim.x;
    for (int64_t t = blockIdx.x; t < n && t < from; t += all)
        for (int c = threadIdx.x; c < m; c += blockDim.x) y[t * ldy + c] = 0;
    for (int64_t t = (to > 0 ? to : 0) + blockIdx.x; t < n; t += all)
        for (int c = threadIdx.x; c < m; c += blockDim.x) y[t * ldy + c] = 0;
}

struct GemmArgs {
    const uint8_t *w, *x;
    const float *ws, *xs;
    int64_t ldw, ldx, ldxs;
    int64_t n;
    int m, k, blocks;                            // result columns, contraction, its blocks
    const int32_t *offsets;
    int groups, m_tiles, total;
    uint16_t *y;
    int64_t ldy;
};

// ---- tiles ----
// A workgroup computes BM columns of y by BN rows.  Slices of one block of k pass through RING
// places in shared memory, loaded straight into them, with the x scales of each wave's rows
// behind them.  The swizzle that spreads rows over the banks is in which piece a lane fetches:
// slot s of row r holds piece s ^ (r & 7).
// TR: W is contracted over its rows.  A slice is 128 rows of W by BM bytes, and the operand is
// turned as it is read.
template <int BM, int BN, int WM, int WN, int RING, bool BF, bool TR>
__global__ void __launch_bounds__(64 * WM * WN)
block_gemm_kernel(GemmArgs p) {
    constexpr int kThreads = 64 * WM * WN, SM = BM / WM, SN = BN / WN, TM = SM / 16, TN = SN / 16;
    constexpr int kPiecesW = BM * 8 / kThreads, kPiecesX = BN * 8 / kThreads;
    constexpr int kPieces = kPiecesW + kPiecesX;
    constexpr int kLoads = kPieces + 1;                   // a slice's loads a wave
    constexpr int kSlice = (BM + BN) * kBlock, kScales = WM * WN * 64;
    constexpr int kPitch = SM * 2 + 16;                   // bytes a row of y takes in the epilogue
    static_assert(SN <= 64 && SM <= 128 && 128 % SM == 0, "a wave's scales");
    static_assert(WM * WN * 16 * kPitch <= RING * kSlice, "the epilogue fits the ring");
    __shared__ __align__(16) uint8_t ring[RING * kSlice];
    __shared__ float scales[RING * kScales];
    const int lane = threadIdx.x & 63, wv = wave_number();
    const int r = lane & 15, g = lane >> 4, wm = wv % WM, wn = wv / WM;
    int total = p.total;
    if (p.offsets) {
        clear_rows_of_no_group(p.offsets, p.groups, p.n, p.y, p.ldy, p.m);
        total = count_tiles(p.offsets, 0, p.groups, p.n, BN, total / p.m_tiles) * p.m_tiles;
        if ((int)blockIdx.x >= total) return;             // fewer tiles than the grid allows for
    }
    // each die takes a run of tiles, in panels eight tiles wide, so that the tiles it works on at
    // a time share their operands in its cache in both directions
    int id = tile_of_die(blockIdx.x, total);
    const int n_tiles = total / p.m_tiles, panel = id / (8 * n_tiles);
    const int wide = p.m_tiles - 8 * panel < 8 ? p.m_tiles - 8 * panel : 8;
    id -= 8 * panel * n_tiles;
    const int mt = 8 * panel + id % wide;
    int nt = id / wide, e = 0;
    int64_t lo = 0, hi = p.n;
    if (p.offsets) {
        e = group_of_tile(p.offsets, 0, p.groups, p.n, BN, nt);
        if (e < 0) return;
        group_rows(p.offsets, e, p.n, lo, hi);
    }
    const int64_t row0 = lo + (int64_t)nt * BN;
    const int m0 = mt * BM + wm * SM;
    // the tile's operands
    const int w_rows = TR ? p.k : p.m;
    const uint8_t *w_at = p.w + (int64_t)e * w_rows * p.ldw + (TR ? mt * BM : (int64_t)mt * BM * p.ldw);
    const uint8_t *x_at = p.x + row0 * p.ldx;
    int64_t piece_at[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const int q = (i < kPiecesW ? i : i - kPiecesW) * kThreads + threadIdx.x;
        if (i < kPiecesW && TR) {
            const int row = q / (BM / 16), s = q % (BM / 16);
            const int left = (int)p.ldw - mt * BM - 16;  // past the edge: repeats, not stored
            const int c = s * 16;
            piece_at[i] = (int64_t)row * p.ldw + (c < left ? c : left);
        } else if (i < kPiecesW) {
            const int row = q >> 3, kp = ((q & 7) ^ (row & 7)) * 16;
            const int left = p.m - mt * BM - 1;
            piece_at[i] = (int64_t)(row < left ? row : left) * p.ldw + kp;
        } else {
            const int row = q >> 3, kp = ((q & 7) ^ (row & 7)) * 16;
            const int64_t left = hi - row0 - 1;
            piece_at[i] = (row < left ? row : left) * p.ldx + kp;
        }
    }
    const float *xs_at;
    {
        const int64_t t = row0 + wn * SN + lane % SN, last = hi - 1;
        xs_at = p.xs + (t < last ? t : last);
    }
    // W's scale of this wave's columns of y
    const int m_block = (m0 < p.m ? m0 : p.m - 1) / kBlock;
    const int w_blocks = blocks_of(TR ? p.m : p.k);       // scales a row of them
    const float *ws_at = p.ws + (int64_t)e * blocks_of(p.m) * blocks_of(p.k) +
                         (TR ? m_block : (int64_t)m_block * w_blocks);
    const int ws_step = TR ? w_blocks : 1;
    auto load_slice = [&](int s) {
        const int b = s < p.blocks ? s : p.blocks - 1;    // the last is repeated, not used
        uint8_t *to = ring + (s % RING) * kSlice;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int q = i < kPiecesW ? i : BM * 8 / kThreads + i - kPiecesW;
            const uint8_t *from;
            if (i < kPiecesW && TR) {
                // rows past the contraction's end meet codes of zero: repeats
                const int row = (i * kThreads + threadIdx.x) / (BM / 16);
                const int over = b * kBlock + row - (p.k - 1);
                from = w_at + piece_at[i] + (int64_t)(b * kBlock - (over > 0 ? over : 0)) * p.ldw;
            } else {
                from = (i < kPiecesW ? w_at : x_at) + piece_at[i] + b * kBlock;
            }
            load_to_lds(from, to + (q * kThreads + wv * 64) * 16);
        }
        load4_to_lds(xs_at + (int64_t)b * p.ldxs, scales + (s % RING) * kScales + wv * 64);
    };
    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int s = 0; s < RING - 1; ++s) load_slice(s);
    for (int s = 0; s < p.blocks; ++s) {
        wait_loads<(RING - 2) * kLoads>();
        barrier_in_place();                               // slice s is there, s - 1 is used up
        load_slice(s + RING - 1);
        const uint8_t *at = ring + (s % RING) * kSlice;
        const uint8_t *xa = at + BM * kBlock + (wn * SN + r) * kBlock;
        const float wscale = ws_at[(int64_t)s * ws_step];
        Operand b[TN];
        float f[TN];
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            b[j].a = *reinterpret_cast<const u32x4 *>(xa + 16 * j * kBlock + (g ^ (r & 7)) * 16);
            b[j].b = *reinterpret_cast<const u32x4 *>(xa + 16 * j * kBlock + ((4 + g) ^ (r & 7)) * 16);
            f[j] = scales[(s % RING) * kScales + wv * 64 + 16 * j + r] * wscale;
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            Operand a;
            if (TR) {
                const uint8_t *wa = at + wm * SM + 16 * i + (r & 1) * 8;
                u32x2 t[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    t[q] = read_turned8(wa + (16 * g + 64 * (q >> 1) + 8 * (q & 1) + (r >> 1)) * BM);
                a.a = u32x4{t[0][0], t[0][1], t[1][0], t[1][1]};
                a.b = u32x4{t[2][0], t[2][1], t[3][0], t[3][1]};
            } else {
                const uint8_t *wa = at + (wm * SM + 16 * i + r) * kBlock;
                a.a = *reinterpret_cast<const u32x4 *>(wa + (g ^ (r & 7)) * 16);
                a.b = *reinterpret_cast<const u32x4 *>(wa + ((4 + g) ^ (r & 7)) * 16);
            }
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const f32x4 z = block_product(a, b[j]);
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[i][j][c] = __builtin_fmaf(z[c], f[j], acc[i][j][c]);
            }
        }
    }
    // 16 rows of y at a time through the wave's part of the ring, so that whole lines are written
    wait_loads<0>();
    __syncthreads();
    const int64_t t0 = row0 + wn * SN;
    uint8_t *out = ring + wv * 16 * kPitch;
    constexpr int kPer = SM / 8;                          // 16-byte pieces a row
#pragma unroll
    for (int j = 0; j < TN; ++j) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
            *reinterpret_cast<uint2 *>(out + r * kPitch + (16 * i + 4 * g) * 2) =
                uint2{Act<BF>::store2(acc[i][j][0], acc[i][j][1]),
                      Act<BF>::store2(acc[i][j][2], acc[i][j][3])};
#pragma unroll
        for (int q = 0; q < (16 * kPer + 63) / 64; ++q) {
            const int piece = q * 64 + lane, row = piece / kPer, c = piece % kPer * 8;
            const int64_t tok = t0 + 16 * j + row;
            if (piece >= 16 * kPer || tok >= hi || m0 + c >= p.m) continue;
            const u32x4 o = *reinterpret_cast<const u32x4 *>(out + row * kPitch + c * 2);
            uint16_t *yo = p.y + tok * p.ldy + m0 + c;
            const int left = p.m - m0 - c;
            if (left >= 8) {
                *reinterpret_cast<u32x4u *>(yo) = o;
            } else {
                for (int v = 0; v < left; ++v) yo[v] = (uint16_t)(o[v >> 1] >> (16 * (v & 1)));
            }
        }
    }
}

}  // namespace

hipError_t launch_block_gemm(const BlockWeightArgs &w, const BlockProductArgs &a, bool bf16,
                             int n_cu, hipStream_t stream) {
    (void)n_cu;
    GemmArgs p{};
    p.w = w.q;
    p.ws = w.scale;
    p.ldw = w.ld;
    p.x = a.x.q;
    p.xs = a.x.scale;
    p.ldx = a.x.ld;
    p.ldxs = a.x.lds;
    p.n = a.n;
    p.m = a.transposed ? w.cols : w.rows;
    p.k = a.transposed ? w.rows : w.cols;
    p.blocks = blocks_of(p.k);
    p.offsets = a.offsets;
    p.groups = w.groups;
    p.y = static_cast<uint16_t *>(a.y);
    p.ldy = a.ldy;
#define EXL3_BLOCK_T(BM, BN, WM, WN, RING, BF, TR)                                             \
    hipLaunchKernelGGL((block_gemm_kernel<BM, BN, WM, WN, RING, BF, TR>),                      \
                       dim3((unsigned)p.total), dim3(64 * WM * WN), 0, stream, p)
#define EXL3_BLOCK(BM, BN, WM, WN, RING)                                                       \
    do {                                                                                       \
        p.m_tiles = (p.m + BM - 1) / BM;                                                       \
        p.total = (int)(p.m_tiles * (a.offsets ? a.n / BN + w.groups : (a.n + BN - 1) / BN));  \
        if (bf16 && a.transposed)                                                              \
            EXL3_BLOCK_T(BM, BN, WM, WN, RING, true, true);                                    \
        else if (bf16)                                                                         \
            EXL3_BLOCK_T(BM, BN, WM, WN, RING, true, false);                                   \
        else if (a.transposed)                                                                 \
            EXL3_BLOCK_T(BM, BN, WM, WN, RING, false, true);                                   \
        else                                                                                   \
            EXL3_BLOCK_T(BM, BN, WM, WN, RING, false, false);                                  \
    } while (0)
    EXL3_BLOCK(128, 128, 2, 2, 2);
#undef EXL3_BLOCK
#undef EXL3_BLOCK_T
    return hipGetLastError();
}

}  // namespace exl3
