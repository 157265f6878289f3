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

#include <algorithm>

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

// ---- few rows ----
// A workgroup takes 16 rows of W, its waves the blocks of the contraction in turn, so that
// neighbouring waves read neighbouring lines; what they hold of W goes from memory straight into
// operands, CH blocks at a time in NB sets.  Rows of x meet it 16 TN at a time, and the waves' sums are added in
// order through shared memory.
// OWN: x comes in 16 bits and each workgroup writes the rows it needs as blocks in shared memory
// (P rows at a time, as fit), while its first loads of W are on their way.
struct RowsKernelArgs {
    GemmArgs p;
    const uint16_t *x16;
    int64_t ldx16;
    int own_rows;                                // OWN: rows a pass
};
template <int TN, int WAVES, int CH, int NB, bool BF, bool OWN>
__global__ void __launch_bounds__(64 * WAVES)
block_rows_kernel(RowsKernelArgs a) {
    const GemmArgs &p = a.p;
    constexpr int kTok = 16 * TN;
    __shared__ float part[WAVES][kTok][16];
    extern __shared__ __align__(16) uint8_t own[];
    const int lane = threadIdx.x & 63, wv = wave_number();
    const int r = lane & 15, g = lane >> 4;
    if (p.offsets) clear_rows_of_no_group(p.offsets, p.groups, p.n, p.y, p.ldy, p.m);
    const int e = blockIdx.x / p.m_tiles, mt = blockIdx.x - e * p.m_tiles;
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
    const int take = OWN ? a.own_rows : kTok;    // rows of x a pass
    constexpr int XB = OWN ? 1 : NB;             // of shared memory nothing is held ahead
    Operand w[NB][CH], x[XB][OWN ? 1 : CH][TN];
    float xs[XB][OWN ? 1 : CH][TN];
    auto load_w = [&](int at, int s0) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            int b = (s0 + c) * WAVES + wv;
            b = b < p.blocks ? b : p.blocks - 1;
            const u32x4 *from = reinterpret_cast<const u32x4 *>(w_at + (int64_t)b * kBlock);
            w[at][c].a = from[0];
            w[at][c].b = from[4];
        }
    };
    for (int64_t t0 = lo; t0 < hi; t0 += take) {
        const int here = (int)(hi - t0 < take ? hi - t0 : take);
        auto load_x1 = [&](int b, Operand (&xo)[TN], float (&so)[TN]) {
            b = b < p.blocks ? b : p.blocks - 1;
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int t = 16 * j + r < here ? 16 * j + r : here - 1;
                const uint8_t *xp = OWN ? own + t * pitch + b * kBlock + 16 * g
                                        : p.x + (t0 + t) * p.ldx + (int64_t)b * kBlock + 16 * g;
                xo[j].a = *reinterpret_cast<const u32x4 *>(xp);
                xo[j].b = *reinterpret_cast<const u32x4 *>(xp + 64);
                so[j] = OWN ? own_scale[b * a.own_rows + t] : p.xs[(int64_t)b * p.ldxs + t0 + t];
            }
        };
        auto load_x = [&](int at, int s0) {
            if (!OWN)
#pragma unroll
                for (int c = 0; c < CH; ++c) load_x1((s0 + c) * WAVES + wv, x[at][c], xs[at][c]);
        };
        load_x(0, 0);
        load_w(0, 0);
        if (OWN) {
            const int pieces = p.blocks * (kBlock / kWide);
            if (t0 != lo) __syncthreads();       // the last pass has read its codes
            for (int i = threadIdx.x; i < here * pieces; i += 64 * WAVES) {
                const int t = i / pieces, c = (i - t * pieces) * kWide;
                float f[kWide];
                widen<BF>(load8(a.x16 + (t0 + t) * a.ldx16 + c, p.k - c), f);
                const CodeScale s = code_scale(largest_of_block(largest8(f)));
                *reinterpret_cast<u32x2 *>(own + t * pitch + c) = to_codes(f, s);
                if ((c & (kBlock - 1)) == 0) own_scale[(c / kBlock) * a.own_rows + t] = s.scale;
            }
            __syncthreads();
        }
        f32x4 acc[TN];
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        auto products = [&](int at, int s0) {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int b = (s0 + c) * WAVES + wv;
                if (b >= p.blocks) continue;     // the same for the whole wave
                const float ws = ws_at[b];
                if (OWN) load_x1(b, x[0][0], xs[0][0]);
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const int ax = OWN ? 0 : at, cx = OWN ? 0 : c;
                    const f32x4 z = block_product(w[at][c], x[ax][cx][j]);
                    const float f = xs[ax][cx][j] * ws;
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[j][i] = __builtin_fmaf(z[i], f, acc[j][i]);
                }
            }
        };
        for (int s = 0; s < steps; s += NB * CH) {
            if (NB == 2 && s + CH < steps) {
                load_x(NB - 1, s + CH);
                load_w(NB - 1, s + CH);
            }
            products(0, s);
            if (s + NB * CH < steps) {
                load_x(0, s + NB * CH);
                load_w(0, s + NB * CH);
            }
            if (NB == 2 && s + CH < steps) products(NB - 1, s + CH);
        }
        if (t0 != lo) __syncthreads();           // the last pass's sums have been read
#pragma unroll
        for (int j = 0; j < TN; ++j)
            *reinterpret_cast<f32x4 *>(&part[wv][16 * j + r][4 * g]) = acc[j];
        __syncthreads();
        for (int i = threadIdx.x; i < kTok * 16; i += 64 * WAVES) {
            const int t = i / 16, m = i % 16;
            float sum = part[0][t][m];
#pragma unroll
            for (int v = 1; v < WAVES; ++v) sum += part[v][t][m];
            if (t < here && m0 + m < p.m) p.y[(t0 + t) * p.ldy + m0 + m] = Act<BF>::store(sum);
        }
    }
}

}  // namespace

namespace {

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
                             int n_cu, hipStream_t stream) {
    RowsKernelArgs r{};
    r.p = gemm_args(w, a);
    r.p.m_tiles = (r.p.m + 15) / 16;
    r.x16 = static_cast<const uint16_t *>(a.x16);
    r.ldx16 = a.ldx16;
    const int64_t total = (int64_t)r.p.m_tiles * w.groups;
    const int64_t avg = (a.n + w.groups - 1) / w.groups;
    (void)n_cu;
    size_t shared = 0;
    if (a.x16) {
        const size_t row = (size_t)r.p.blocks * kBlock + 16 + (size_t)r.p.blocks * 4;
        r.own_rows = (int)std::min<size_t>(16, std::max<size_t>(1, kOwnBytes / row));
        shared = r.own_rows * row;
    }
#define EXL3_ROWS_T(TN, WAVES, CH, NB, BF, OWN)                                                 \
    hipLaunchKernelGGL((block_rows_kernel<TN, WAVES, CH, NB, BF, OWN>), dim3((unsigned)total),  \
                       dim3(64 * WAVES), shared, stream, r)
#define EXL3_ROWS(TN, WAVES, CH, NB, OWN)                  \
    do {                                                   \
        if (bf16)                                          \
            EXL3_ROWS_T(TN, WAVES, CH, NB, true, OWN);     \
        else                                               \
            EXL3_ROWS_T(TN, WAVES, CH, NB, false, OWN);    \
    } while (0)
    // The waves and what each has under way, by the contraction's blocks, us:
    //   16 blocks (64 experts of 1408 x 2048, 64 rows): 8 waves of two blocks 25, 8 of four 47,
    //   16 of two 43 (idle waves still take their places)
    //   32 (12288 x 4096, 1 row, own): 8 of four 12.1, 16 of two 12.5, 8 of two 16.6; 16 rows:
    //   16.4, 13.5 and 15.9
    //   96 (4096 x 12288, 16 rows): 16 of two 14.0, 8 of four 14.4, 8 of two 15.0
    const int blocks = r.p.blocks;
    if (a.x16) {
        if (blocks <= 16)
            EXL3_ROWS(1, 8, 2, 1, true);
        else if (blocks <= 32)
            EXL3_ROWS(1, 8, 4, 1, true);
        else
            EXL3_ROWS(1, 16, 2, 1, true);
    } else if (avg <= 16) {
        if (blocks <= 16)
            EXL3_ROWS(1, 8, 2, 1, false);
        else
            EXL3_ROWS(1, 16, 2, 1, false);
    } else {
        EXL3_ROWS(2, 8, 1, 2, false);
    }
#undef EXL3_ROWS
#undef EXL3_ROWS_T
    return hipGetLastError();
}

hipError_t launch_block_gemm(const BlockWeightArgs &w, const BlockProductArgs &a, bool bf16,
                             int n_cu, hipStream_t stream) {
    (void)n_cu;
    GemmArgs p = gemm_args(w, a);
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
