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
//
// The unit aligns the products of eight neighbouring k's to the largest and keeps 13 bits below its
// leading one (measured: 2^16 + 2^s is exact from s = 3 on within such an eight, and to 24 bits
// across them); the rest is binary32.  With the loss of that emulated, 4,096 normally distributed
// terms are off by 2e-5 (root mean square; 3.7e-5 where some channels are 12 times the others, 1e-4
// where 200 times), rounding the result to binary16 takes 2.1e-4 and to bfloat16 1.7e-3.  It is the
// price of the 8-bit rate: codes widened to bfloat16 run at half of it.
#include "blocks.h"

#include <algorithm>

namespace exl3 {

namespace {

using i32x8 = int __attribute__((ext_vector_type(8)));

struct Operand {
    u32x4 a, b;                                  // pieces g and 4 + g
};
// A scale as mantissa * 2^(exponent - 127), for where a block's factor, the product of its two
// scales, is out of range though what it meets may bring it back: the instruction takes the
// exponents, and the mantissas' product is the factor.  NaN and infinity give NaN; zero and
// subnormal scales have the least exponent.
struct Scale {
    float mantissa;
    int exponent;
};
__device__ __forceinline__ Scale split_scale(float s) {
    const int e = __builtin_bit_cast(uint32_t, s) >> 23 & 255;
    return Scale{__builtin_ldexpf(s, 127 - e), e};
}
template <bool SCALED>
__device__ __forceinline__ f32x4 block_product(const Operand &w, const Operand &x,
                                               int w_exponent = 0, int x_exponent = 0) {
    i32x8 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[i] = (int)w.a[i];
        a[4 + i] = (int)w.b[i];
        b[i] = (int)x.a[i];
        b[4 + i] = (int)x.b[i];
    }
    // both formats e4m3; scales of one, or each lane's exponents in the lowest byte
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    if (SCALED)
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, w_exponent, 0,
                                                                x_exponent);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, 0, 0, 0);
}

// Turns 8 x 16 bytes: of 16 lanes, lane 2 j + q names bytes 8 q .. 8 q + 7 of row j, and lane i
// gets byte i of rows 0..7.
using i32x2 = int __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u32x2 read_turned8(const uint8_t *from) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32(
        (__attribute__((address_space(3))) i32x2 *)from));
}

// 16 (or four) bytes a lane straight into shared memory, at to + 16 (4) lane, from a uniform base
// and a lane's offset.  Written out because the compiler, which knows what its own form of it
// writes, waits for all such loads under way before the next read of shared memory; here the
// caller's wait_loads and barriers order them.  (The move to m0 needs one state before its use.)
__device__ __forceinline__ void stage16(const uint8_t *base, uint32_t offset, uint32_t to) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :: "v"(offset), "s"(base), "s"(to) : "memory");
}
__device__ __forceinline__ void stage4(const float *base, uint32_t offset, uint32_t to) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
                 :: "v"(offset), "s"(base), "s"(to) : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void *p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void *)p;
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
// A workgroup computes BM columns of y by BN rows, each wave SM x SN of them.  Slices of one block
// of k pass through RING places in shared memory, loaded straight into them, with the x scales of
// each wave's rows behind them.  The swizzle that spreads rows over the banks is in which piece a
// lane fetches: slot s of row r holds piece s ^ (r & 7).
// While the matrix units work on 16 rows of W, the next 16 are read and the results before are
// scaled and added.  The one barrier a slice stands where its last rows have just been read: its
// place is free for the slice RING later, and the next slice is there.
// TR: W is contracted over its rows.  A slice is 128 rows of W by BM bytes, and the operand is
// turned as it is read: 16 lanes read eight rows of 16 bytes, and turned_slot puts the rows that a
// wave's 32 lanes read at a time into different banks.
// WK: sets of waves with rings of their own that take the contraction's blocks by turns, for calls
// of few tiles; their sums are added in order.
// 4,096 rows, 12288 x 4096: 166 to 185 us by the card, 2.23 to 2.48 PFLOP/s; 176 on one where the
// library's product with one scale for each operand took 173 to 175.  Matrix units are busy 66 % of
// a compute unit's busy cycles (59 % of the kernel's), vector instructions issued on 53 %, shared
// memory active on 31 %; turned, 2,000 rows, 4096 x 4096: 49, 48 and 30 %; 128 x 64 tiles, 333 rows:
// 30, 36 and 28 %, with waves waiting for 38 % of theirs.
// 24 rows, 4096 x 12288: 11.6 us, 4.3 TB/s (32 x 32 tiles, four sets).
template <int BM>
__device__ __forceinline__ int turned_slot(int row) {
    constexpr int kSame = BM == 256 ? 1 : BM == 128 ? 2 : BM == 64 ? 4 : 8;   // rows in 256 bytes
    return (row & 7) / kSame | (row >> 4 & 1) * (8 / kSame);
}

template <int BM, int BN, int WM, int WN, int WK, int RING, int SPREAD, bool BF, bool TR>
__global__ void __launch_bounds__(64 * WM * WN * WK)
block_gemm_kernel(const uint8_t *__restrict__ w, const float *__restrict__ w_scale,
                  const uint8_t *__restrict__ x, const float *__restrict__ x_scale,
                  const int32_t *__restrict__ offsets, uint16_t *__restrict__ y, GemmArgs p) {
    constexpr int kThreads = 64 * WM * WN, SM = BM / WM, SN = BN / WN, TM = SM / 16, TN = SN / 16;
    constexpr int kPiecesW = BM * 8 / kThreads, kPiecesX = BN * 8 / kThreads;
    constexpr int kPieces = kPiecesW + kPiecesX;
    constexpr int kLoads = kPieces + 1;                   // a slice's loads a wave
    constexpr int kScales = (BM + BN) * kBlock, kSlice = kScales + WM * WN * 64 * 4;
    constexpr int kSpread = SPREAD, kSlots = kSpread * TN;
    constexpr float kLift = 0x1p24f;                      // what the factors are multiplied by
    constexpr int kPitch = SM * 2 + 16;                   // bytes a row of y takes in the epilogue
    static_assert(SN <= 64 && SM <= 128 && 128 % SM == 0, "a wave's scales");
    static_assert(SPREAD < TM || (SPREAD == TM && RING > 2), "a slice's loads precede its wait");
    static_assert(TM % 2 == 0, "two places for rows of W");
    static_assert((WK - 1) * BM * BN * 4 + WM * WN * 16 * kPitch <= WK * RING * kSlice,
                  "the sets' sums and the epilogue fit the rings");
    __shared__ __align__(16) uint8_t rings[WK * RING * kSlice + WK * WM * WN * 256];
    const int lane = threadIdx.x & 63, wk = WK == 1 ? 0 : wave_number() / (WM * WN);
    const int wv = WK == 1 ? wave_number() : wave_number() % (WM * WN);
    const int tid = WK == 1 ? (int)threadIdx.x : (int)threadIdx.x % (64 * WM * WN);
    uint8_t *ring = rings + wk * RING * kSlice;           // this set's
    const int r = lane & 15, g = lane >> 4, wm = wv % WM, wn = wv / WM;
    int total = p.total;
    if (offsets) {
        clear_rows_of_no_group(offsets, p.groups, p.n, y, p.ldy, p.m);
        total = count_tiles(offsets, 0, p.groups, p.n, BN, total / p.m_tiles) * p.m_tiles;
        total = __builtin_amdgcn_readfirstlane(total);    // all lanes have the same
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
    if (offsets) {
        e = group_of_tile(offsets, 0, p.groups, p.n, BN, nt);
        if (e < 0) return;
        e = __builtin_amdgcn_readfirstlane(e);
        nt = __builtin_amdgcn_readfirstlane(nt);
        group_rows(offsets, e, p.n, lo, hi);
    }
    const int64_t row0 = lo + (int64_t)nt * BN;
    const int m0 = mt * BM + wm * SM;
    // this set's blocks: first, first + WK, .. (a set without any computes with factors of zero)
    const int first = wk < p.blocks ? wk : 0, steps = (p.blocks + WK - 1) / WK;
    // the tile's operands from uniform bases that move along k, and 32-bit offsets of the
    // thread's pieces
    const int w_rows = TR ? p.k : p.m;
    const uint8_t *w_at = w + (int64_t)e * w_rows * p.ldw +
                          (TR ? mt * BM + (int64_t)first * kBlock * p.ldw
                              : (int64_t)mt * BM * p.ldw + first * kBlock);
    const uint8_t *x_at = x + row0 * p.ldx + first * kBlock;
    const float *xs_at = x_scale + row0 + first * p.ldxs;
    uint32_t xs_lane;                                     // this lane's row of them
    {
        const int64_t t = wn * SN + lane % SN, last = hi - 1 - row0;
        xs_lane = (uint32_t)(t < last ? t : last) * 4;
    }
    uint32_t piece_at[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const int q = (i < kPiecesW ? i : i - kPiecesW) * kThreads + tid;
        const int row = i < kPiecesW && TR ? q / (BM / 16) : q >> 3;
        if (i < kPiecesW && TR) {
            const int c = ((q % (BM / 16)) ^ turned_slot<BM>(row)) * 16;
            const int left = (int)p.ldw - mt * BM - 16;   // past the edge: repeats, not stored
            piece_at[i] = (uint32_t)row * (uint32_t)p.ldw + (uint32_t)(c < left ? c : left);
        } else {
            const int kp = ((q & 7) ^ (row & 7)) * 16;
            const int64_t left = i < kPiecesW ? p.m - mt * BM - 1 : hi - row0 - 1;
            piece_at[i] = (uint32_t)(row < left ? row : left) *
                              (uint32_t)(i < kPiecesW ? p.ldw : p.ldx) + (uint32_t)kp;
        }
    }
    const uint32_t ring_at = lds_address(ring);
    // the last slice of TR: rows past the contraction's end meet codes of zero and repeat its last
    const int short_by = TR ? p.blocks * kBlock - p.k : 0;
    auto load_piece = [&](int i, int b, int place) {
        const int q = i < kPiecesW ? i : BM * 8 / kThreads + i - kPiecesW;
        uint32_t at = piece_at[i];
        if (TR && i < kPiecesW && short_by && b >= p.blocks - 1) {
            const int row = (i * kThreads + tid) / (BM / 16);
            const int over = row - (kBlock - 1 - short_by);
            at -= (uint32_t)(over > 0 ? over : 0) * (uint32_t)p.ldw;
        }
        stage16(i < kPiecesW ? w_at : x_at, at,
                ring_at + place * kSlice + (q * kThreads + wv * 64) * 16);
    };
    auto load_scales = [&](int place) {
        stage4(xs_at, xs_lane, ring_at + place * kSlice + kScales + wv * 256);
    };
    auto read_scale = [&](int j, int place) {
        return *reinterpret_cast<const float *>(ring + place * kSlice + kScales + wv * 256 +
                                                (16 * j + r) * 4);
    };
    // from the slice of step s to the next; the last is repeated into places that nobody reads
    auto advance = [&](int s) {
        if (wk + WK * (s + 1) >= p.blocks) return;
        w_at += TR ? (int64_t)WK * kBlock * p.ldw : WK * kBlock;
        x_at += WK * kBlock;
        xs_at += WK * p.ldxs;
    };
    // W's scales of this wave's columns of y
    const int m_block = (m0 < p.m ? m0 : p.m - 1) / kBlock;
    // 64 steps' at a time, a step's in a lane: a scalar load is one that each wait for shared
    // memory would wait for, some 400 cycles (0 for a step past the last).  The first come with
    // the slices' loads, so that nothing waits for all of these.
    const float *ws_at = w_scale + (int64_t)e * blocks_of(p.m) * p.blocks +
                         (TR ? m_block : (int64_t)m_block * p.blocks);
    auto w_scale_of = [&](int c) { return ws_at[TR ? (int64_t)c * blocks_of(p.m) : c]; };
    auto w_place = [&](int s) {                           // of step s + lane, in bytes
        const int now = wk + WK * (s + lane);
        return (uint32_t)(now < p.blocks ? now : 0) * (TR ? (uint32_t)blocks_of(p.m) * 4u : 4u);
    };
    auto w_there = [&](int s, float v) { return wk + WK * (s + lane) < p.blocks ? v : 0.0f; };
    const int w_first = WK * RING * kSlice + (wk * WM * WN + wv) * 256;
    stage4(ws_at, w_place(0), lds_address(rings) + w_first);
    auto of_lane = [](float v, int l) {
        return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
    };
    Operand a[2], b[TN];
    float f[TN], f_last[TN];
    f32x4 acc[TM][TN], z[2][TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        f_last[j] = 0.0f;
        z[1][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < TM; ++i) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const int at_a = (g ^ (r & 7)) * 16, at_b = ((4 + g) ^ (r & 7)) * 16;
    auto read_a = [&](int i, int place, Operand &to) {
        const uint8_t *at = ring + place * kSlice;
        if (TR) {
            u32x2 t[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int row = 16 * g + 64 * (q >> 1) + 8 * (q & 1) + (r >> 1);
                const int slot = (wm * (SM / 16) + i) ^ turned_slot<BM>(row);
                t[q] = read_turned8(at + row * BM + slot * 16 + (r & 1) * 8);
            }
            to.a = u32x4{t[0][0], t[0][1], t[1][0], t[1][1]};
            to.b = u32x4{t[2][0], t[2][1], t[3][0], t[3][1]};
        } else {
            const uint8_t *wa = at + (wm * SM + 16 * i + r) * kBlock;
            to.a = *reinterpret_cast<const u32x4 *>(wa + at_a);
            to.b = *reinterpret_cast<const u32x4 *>(wa + at_b);
        }
    };
    auto read_b = [&](int j, int place, Operand &to) {
        const uint8_t *xa = ring + place * kSlice + (BM + wn * SN + 16 * j + r) * kBlock;
        to.a = *reinterpret_cast<const u32x4 *>(xa + at_a);
        to.b = *reinterpret_cast<const u32x4 *>(xa + at_b);
    };
    auto scale_add = [&](int i, int j, float by) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            acc[i][j][c] = __builtin_fmaf(z[i & 1][j][c], by, acc[i][j][c]);
    };
    // A slice's loads go out one after the other over kSpread rows of matrix instructions: all at
    // once they wait for one another, and the wave with them.
    auto load_slot = [&](int slot, int s, int place) {
#pragma unroll
        for (int q = 0; q < kLoads; ++q)
            if (q * kSlots / kLoads == slot) {
                if (q < kPieces)
                    load_piece(q, wk + WK * s, place);
                else
                    load_scales(place);
            }
    };
#pragma unroll
    for (int s = 0; s < RING; ++s) {
#pragma unroll
        for (int slot = 0; slot < (s + 1 < RING ? kSlots : TN); ++slot) load_slot(slot, s, s);
        if (s + 1 < RING || kSpread == 1) advance(s);
    }
    wait_loads<(RING - 2) * kLoads + (kLoads * TN + kSlots - 1) / kSlots>();
    barrier_in_place();
    float w64 = kLift * w_there(0, *reinterpret_cast<const float *>(rings + w_first + lane * 4));
    const float ws = of_lane(w64, 0);
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        read_b(j, 0, b[j]);
        f[j] = read_scale(j, 0) * ws;
    }
    read_a(0, 0, a[0]);
    int place = 0, before = RING - 1;
    for (int s0 = 0; s0 < steps; s0 += 63) {              // a step takes the next one's scale
        if (s0)
            w64 = kLift * w_there(s0, *reinterpret_cast<const float *>(
                                          reinterpret_cast<const char *>(ws_at) + w_place(s0)));
        for (int s = s0; s < steps && s < s0 + 63; ++s) {
            const int after = place + 1 == RING ? 0 : place + 1;
#pragma unroll
            for (int i = 0; i < TM; ++i) {
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    __builtin_amdgcn_sched_barrier(0);
                    z[i & 1][j] = block_product<false>(a[i & 1], b[j]);
                    __builtin_amdgcn_sched_barrier(0);
                    // under the matrix instructions: the next operands, the results before and loads
                    if (j == 0 && i + 1 < TM) read_a(i + 1, place, a[(i + 1) & 1]);
                    if (i + 1 == TM) {
                        if (j == 0) read_a(0, after, a[0]);         // the next slice's
                        read_b(j, after, b[j]);
                        load_slot(j, s + RING, place);
                    } else if (i + 1 < kSpread) {
                        load_slot((i + 1) * TN + j, s - 1 + RING, before);
                    }
                    if (i == 0)
                        scale_add(TM - 1, j, f_last[j]);
                    else
                        scale_add(i - 1, j, f[j]);
                    if (i + 1 == TM) {
                        f_last[j] = f[j];
                        f[j] = read_scale(j, after);
                    }
                }
                if (i + 2 == kSpread) advance(s + RING - 1);  // the last of its loads is out
                if (kSpread == 1 && i + 1 == TM) advance(s + RING);
                if (i + 2 == TM) {
                    __builtin_amdgcn_sched_barrier(0);
                    wait_loads<(RING - 2) * kLoads>();
                    barrier_in_place();
                }
            }
#pragma unroll
            for (int j = 0; j < TN; ++j) f[j] *= of_lane(w64, s - s0 + 1);
            before = place;
            place = after;
        }
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) scale_add(TM - 1, j, f_last[j]);
    // Factors and sums are held over 2^-24 (kLift): a factor that is subnormal then, the product of
    // two scales below 2^-150, is off by at most 2^-174, and what it meets, less than 2^25, by less
    // than any result shows.  An infinite factor leaves infinity or NaN, whatever it meets.  Where a
    // sum is past the largest number, this wave's sums once more, by the scales' exponents and from
    // memory; not for rows that are NaN by their scales.
    // 4,096 rows, 12288 x 4096, against factors without any of this, in turn on one card: 0.5 % more
    // (163.3 us for 162.5); the exponents carried through the loop 4 %, a second loop that takes
    // them from the first such factor on 1 % (both 8 to 11 % of 1,000 to 2,000 rows, 4096 x 4096).
    uint32_t past = 0;                                    // by rows of 16
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        float sum = 0.0f;                                 // finite if all are, and below 2^63
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int c = 0; c < 4; c += 2)
                sum = __builtin_fmaf(acc[i][j][c], acc[i][j][c + 1], sum);
        past |= !(fabsf(sum) <= FLT_MAX) ? 1u << j : 0;
    }
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][j][c] *= 1.0f / kLift;
    if (__builtin_amdgcn_ballot_w64(past != 0)) {
        const uint8_t *xs_rows = x + row0 * p.ldx;
        bool bad = false;
        for (int c = wk; c < p.blocks; c += WK)
            bad = bad || !(fabsf(x_scale[row0 + (int64_t)c * p.ldxs + xs_lane / 4]) <= FLT_MAX);
        const uint64_t bad_rows = __builtin_amdgcn_ballot_w64(bad);
        bool again = false;
#pragma unroll
        for (int j = 0; j < TN; ++j)
            again = again || (past >> j & 1 && !(bad_rows >> (16 * j + r) & 1));
        if (__builtin_amdgcn_ballot_w64(again)) {
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
            for (int c = wk; c < p.blocks; c += WK) {
                const Scale sw = split_scale(w_scale_of(c));
                int x_exponent[TN];
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    int64_t t = wn * SN + 16 * j + r;
                    t = t < hi - 1 - row0 ? t : hi - 1 - row0;
                    const Scale sx = split_scale(x_scale[row0 + (int64_t)c * p.ldxs + t]);
                    x_exponent[j] = sx.exponent;
                    f[j] = sx.mantissa * sw.mantissa;
                    const u32x4 *from = reinterpret_cast<const u32x4 *>(
                        xs_rows + t * p.ldx + (int64_t)c * kBlock + 16 * g);
                    b[j].a = from[0];
                    b[j].b = from[4];
                }
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    __builtin_amdgcn_sched_barrier(0);
                    const uint8_t *from = w + (int64_t)e * w_rows * p.ldw;
                    const int m = m0 + 16 * i + r;
                    if (TR) {
                        from += m < (int)p.ldw ? m : (int)p.ldw - 1;
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            uint32_t v = 0;
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                int k = c * kBlock + (q >> 2) * 64 + 16 * g + 4 * (q & 3) + h;
                                k = k < p.k ? k : p.k - 1;    // (meets codes of zero)
                                v |= (uint32_t)from[k * p.ldw] << 8 * h;
                            }
                            (q < 4 ? a[0].a : a[0].b)[q & 3] = v;
                        }
                    } else {
                        const u32x4 *at = reinterpret_cast<const u32x4 *>(
                            from + (int64_t)(m < p.m ? m : p.m - 1) * p.ldw + (int64_t)c * kBlock +
                            16 * g);
                        a[0].a = at[0];
                        a[0].b = at[4];
                    }
#pragma unroll
                    for (int j = 0; j < TN; ++j) {
                        z[i & 1][j] = block_product<true>(a[0], b[j], sw.exponent, x_exponent[j]);
                        scale_add(i, j, f[j]);
                    }
                }
            }
        }
    }
    // 16 rows of y at a time through the wave's part of the ring, so that whole lines are written
    wait_loads<0>();
    __syncthreads();
    if constexpr (WK > 1) {
        // the sets' sums, added in order
        f32x4 *sums = reinterpret_cast<f32x4 *>(rings);
        if (wk > 0)
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    sums[((wk - 1) * TM * TN + i * TN + j) * kThreads + tid] = acc[i][j];
        __syncthreads();
        if (wk > 0) return;
#pragma unroll
        for (int v = 1; v < WK; ++v)
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    acc[i][j] += sums[((v - 1) * TM * TN + i * TN + j) * kThreads + tid];
        // (a wave's place in the epilogue lies where sums of any wave were: past them)
    }
    const int64_t t0 = row0 + wn * SN;
    uint8_t *out = rings + (WK - 1) * BM * BN * 4 + wv * 16 * kPitch;
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
            uint16_t *yo = y + tok * p.ldy + m0 + c;
            const int left = p.m - m0 - c;
            if (left >= 8) {
                *reinterpret_cast<u32x4u *>(yo) = o;
            } else {
                for (int v = 0; v < left; ++v) yo[v] = (uint16_t)(o[v >> 1] >> (16 * (v & 1)));
            }
        }
    }
}

// ---- few rows ----
// A workgroup takes 16 rows of W, its waves the blocks of the contraction in turn, so that
// neighbouring waves read neighbouring lines; what they hold of W goes from memory straight into
// operands, CH blocks at a time.  Rows of x meet it 16 at a time, and the waves' sums are added in
// order through shared memory.
// The scales' exponents go into the instruction, as the sums wait for memory (12288 x 4096, 1 row:
// 12.6 us, 12.4 by the scales' product).
// OWN: x comes in 16 bits and each workgroup writes the rows it needs as blocks in shared memory
// (own_rows at a time, as fit), while its first loads of W are on their way.
// 1 row, 12288 x 4096: 12 us, 4.2 TB/s, in one launch; bound by the loads of W, of which all are
// under way at once, and the launch's start and end.
struct RowsKernelArgs {
    GemmArgs p;
    const uint16_t *x16;
    int64_t ldx16;
    int own_rows;                                // OWN: rows a pass
    int group0;                                  // the first of this launch
};
template <int WAVES, int CH, bool BF, bool OWN>
__global__ void __launch_bounds__(64 * WAVES)
block_rows_kernel(RowsKernelArgs a) {
    const GemmArgs &p = a.p;
    __shared__ float part[WAVES][16][16];
    extern __shared__ __align__(16) uint8_t own[];
    const int lane = threadIdx.x & 63, wv = wave_number();
    const int r = lane & 15, g = lane >> 4;
    if (p.offsets) clear_rows_of_no_group(p.offsets, p.groups, p.n, p.y, p.ldy, p.m);
    const int e = a.group0 + blockIdx.x / p.m_tiles, mt = blockIdx.x % p.m_tiles;
    int64_t lo, hi;
    group_rows(p.offsets, e, p.n, lo, hi);
    if (lo >= hi) return;
    const int m0 = mt * 16;
    int wr = m0 + r;
    wr = wr < p.m ? wr : p.m - 1;                // past the edge: repeats, not stored
    const uint8_t *w_at = p.w + ((int64_t)e * p.m + wr) * p.ldw + 16 * g;
    const float *ws_at = p.ws + ((int64_t)e * blocks_of(p.m) + m0 / kBlock) * p.blocks;
    const int steps = (p.blocks + WAVES - 1) / WAVES;
    const int pitch = p.blocks * kBlock + 16;    // OWN: a row of codes in shared memory
    float *own_scale = reinterpret_cast<float *>(own + a.own_rows * pitch);
    const int take = OWN ? a.own_rows : 16;      // rows of x a pass
    Operand w[CH], x[OWN ? 1 : CH];
    float xs[OWN ? 1 : CH];
    auto load_w = [&](int s0) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            int b = (s0 + c) * WAVES + wv;
            b = b < p.blocks ? b : p.blocks - 1;
            const u32x4 *from = reinterpret_cast<const u32x4 *>(w_at + (int64_t)b * kBlock);
            w[c].a = from[0];
            w[c].b = from[4];
        }
    };
    for (int64_t t0 = lo; t0 < hi; t0 += take) {
        const int here = (int)(hi - t0 < take ? hi - t0 : take), t = r < here ? r : here - 1;
        auto load_x1 = [&](int b, Operand &to, float &scale) {
            b = b < p.blocks ? b : p.blocks - 1;
            const uint8_t *xp = OWN ? own + t * pitch + b * kBlock + 16 * g
                                    : p.x + (t0 + t) * p.ldx + (int64_t)b * kBlock + 16 * g;
            to.a = *reinterpret_cast<const u32x4 *>(xp);
            to.b = *reinterpret_cast<const u32x4 *>(xp + 64);
            scale = OWN ? own_scale[b * a.own_rows + t] : p.xs[(int64_t)b * p.ldxs + t0 + t];
        };
        auto load_x = [&](int s0) {              // of shared memory nothing is held ahead
            if (!OWN)
#pragma unroll
                for (int c = 0; c < CH; ++c) load_x1((s0 + c) * WAVES + wv, x[c], xs[c]);
        };
        load_x(0);
        load_w(0);
        if (OWN) {
            const int pieces = p.blocks * (kBlock / kWide);
            if (t0 != lo) __syncthreads();       // the last pass has read its codes
            for (int i = threadIdx.x; i < here * pieces; i += 64 * WAVES) {
                const int row = i / pieces, c = (i - row * pieces) * kWide;
                float f[kWide];
                widen<BF>(load8(a.x16 + (t0 + row) * a.ldx16 + c, p.k - c), f);
                const CodeScale s = code_scale(largest_of_block(largest8(f)));
                *reinterpret_cast<u32x2 *>(own + row * pitch + c) = to_codes(f, s);
                if ((c & (kBlock - 1)) == 0) own_scale[(c / kBlock) * a.own_rows + row] = s.scale;
            }
            __syncthreads();
        }
        f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int s = 0; s < steps; s += CH) {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int b = (s + c) * WAVES + wv, cx = OWN ? 0 : c;
                if (b >= p.blocks) continue;     // the same for the whole wave
                if (OWN) load_x1(b, x[0], xs[0]);
                const Scale fx = split_scale(xs[cx]), fw = split_scale(ws_at[b]);
                const f32x4 z = block_product<true>(w[c], x[cx], fw.exponent, fx.exponent);
                const float f = fx.mantissa * fw.mantissa;
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(z[i], f, acc[i]);
            }
            if (s + CH < steps) {
                load_x(s + CH);
                load_w(s + CH);
            }
        }
        if (t0 != lo) __syncthreads();           // the last pass's sums have been read
        *reinterpret_cast<f32x4 *>(&part[wv][r][4 * g]) = acc;
        __syncthreads();
        if (threadIdx.x < 256) {
            const int row = threadIdx.x / 16, m = threadIdx.x % 16;
            float sum = part[0][row][m];
#pragma unroll
            for (int v = 1; v < WAVES; ++v) sum += part[v][row][m];
            if (row < here && m0 + m < p.m)
                p.y[(t0 + row) * p.ldy + m0 + m] = Act<BF>::store(sum);
        }
    }
}

GemmArgs gemm_args(const BlockWeightArgs &w, const BlockProductArgs &a) {
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
    return p;
}

}  // namespace

hipError_t launch_block_rows(const BlockWeightArgs &w, const BlockProductArgs &a, bool bf16,
                             hipStream_t stream) {
    RowsKernelArgs r{};
    r.p = gemm_args(w, a);
    r.p.m_tiles = (r.p.m + 15) / 16;
    r.x16 = static_cast<const uint16_t *>(a.x16);
    r.ldx16 = a.ldx16;
    size_t shared = 0;
    if (a.x16) {
        const size_t row = (size_t)r.p.blocks * kBlock + 16 + (size_t)r.p.blocks * 4;
        r.own_rows = (int)std::min<size_t>(16, std::max<size_t>(1, kOwnBytes / row));
        shared = r.own_rows * row;
    }
#define EXL3_ROWS_T(WAVES, CH, BF, OWN)                                                          \
    hipLaunchKernelGGL((block_rows_kernel<WAVES, CH, BF, OWN>), dim3(grid), dim3(64 * WAVES),    \
                       shared, stream, r)
#define EXL3_ROWS(WAVES, CH)                   \
    do {                                       \
        if (a.x16 && bf16)                     \
            EXL3_ROWS_T(WAVES, CH, true, true); \
        else if (a.x16)                        \
            EXL3_ROWS_T(WAVES, CH, false, true); \
        else if (bf16)                         \
            EXL3_ROWS_T(WAVES, CH, true, false); \
        else                                   \
            EXL3_ROWS_T(WAVES, CH, false, false); \
    } while (0)
    // The waves and what each has under way, by the contraction's blocks, us:
    //   16 blocks (64 experts of 1408 x 2048, 64 rows): 8 waves of two blocks 25, 8 of four 47,
    //   16 of two 43 (idle waves still take their places)
    //   32 (12288 x 4096, 1 row, own): 8 of four 12.1, 16 of two 12.5, 8 of two 16.6
    //   96 (4096 x 12288, 16 rows): 16 of two 14.0, 8 of four 14.4, 8 of two 15.0
    const int blocks = r.p.blocks;
    // a launch has fewer than 2^32 lanes, of up to 1,024 a workgroup
    const int per = std::max(1, (1 << 21) / r.p.m_tiles);
    for (r.group0 = 0; r.group0 < w.groups; r.group0 += per) {
        const unsigned grid = (unsigned)(r.p.m_tiles * std::min(per, w.groups - r.group0));
        if (blocks <= 16)
            EXL3_ROWS(8, 2);
        else if (blocks <= 32)
            EXL3_ROWS(8, 4);
        else
            EXL3_ROWS(16, 2);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
#undef EXL3_ROWS
#undef EXL3_ROWS_T
    return hipSuccess;
}

hipError_t launch_block_gemm(const BlockWeightArgs &w, const BlockProductArgs &a, BlockForm form,
                             bool bf16, hipStream_t stream) {
    GemmArgs p = gemm_args(w, a);
#define EXL3_BLOCK_T(BM, BN, WM, WN, WK, RING, SPREAD, BF, TR)                                 \
    hipLaunchKernelGGL((block_gemm_kernel<BM, BN, WM, WN, WK, RING, SPREAD, BF, TR>),          \
                       dim3((unsigned)p.total), dim3(64 * WM * WN * WK), 0, stream, p.w, p.ws, \
                       p.x, p.xs, p.offsets, p.y, p)
#define EXL3_BLOCK(BM, BN, WM, WN, WK, RING, SPREAD)                                           \
    do {                                                                                       \
        p.m_tiles = (p.m + BM - 1) / BM;                                                       \
        p.total =                                                                              \
            (int)(p.m_tiles * (a.offsets ? a.n / BN + w.groups : (a.n + BN - 1) / BN));        \
        if (bf16 && a.transposed)                                                              \
            EXL3_BLOCK_T(BM, BN, WM, WN, WK, RING, SPREAD, true, true);                        \
        else if (bf16)                                                                         \
            EXL3_BLOCK_T(BM, BN, WM, WN, WK, RING, SPREAD, true, false);                       \
        else if (a.transposed)                                                                 \
            EXL3_BLOCK_T(BM, BN, WM, WN, WK, RING, SPREAD, false, true);                       \
        else                                                                                   \
            EXL3_BLOCK_T(BM, BN, WM, WN, WK, RING, SPREAD, false, false);                      \
    } while (0)
    switch (form) {
        case kTile256x256: EXL3_BLOCK(256, 256, 2, 4, 1, 2, 4); break;
        case kTile256x128: EXL3_BLOCK(256, 128, 4, 2, 1, 3, 4); break;
        case kTile128x128Twice: EXL3_BLOCK(128, 128, 2, 2, 1, 2, 1); break;
        case kTile128x128: EXL3_BLOCK(128, 128, 2, 2, 1, 4, 4); break;
        case kTile128x64: EXL3_BLOCK(128, 64, 2, 2, 2, 3, 4); break;
        case kTile128x32: EXL3_BLOCK(128, 32, 2, 2, 2, 3, 4); break;
        case kTile64x32: EXL3_BLOCK(64, 32, 1, 1, 4, 3, 4); break;
        case kTile32x32: EXL3_BLOCK(32, 32, 1, 1, 4, 4, 2); break;
        default: return hipErrorInvalidValue;
    }
#undef EXL3_BLOCK
#undef EXL3_BLOCK_T
    return hipGetLastError();
}

}  // namespace exl3
