// Device-side reading of coded weights in the register layout of the matrix
// instructions (gfx950), shared by the products with coded weights.
//
// A matrix instruction contracts 32 values k per step: lane l holds row l & 15
// of its operand and, with g = l >> 4, eight of the 32 k's.  Which k a lane's
// eight are is free as long as both operands agree, so a lane takes one whole
// row of one 16 x 16 tile: of 64 consecutive columns (four tiles), lane group
// g owns tile g, and its row's 16 consecutive trellis positions are the
// operands of two steps: columns 16 g + 0..7, then 16 g + 8..15.  Sixteen
// consecutive positions are one run of 16 K stream bits, and their states are
// windows of that run and the 16 bits before it: K / 2 + 1 words loaded (K
// even; K = 2: two) for 16 weights, no shared memory and no exchange of lanes.
//
// The levels are computed, not looked up: the 128 KiB table would cost every
// compute unit a fill as large as its share of many a matrix's codes, and 64
// random LDS reads of a wave meet in few banks.
//   mul1: h = A s mod 2^32 (one 32-bit product; two 24-bit ones and a shift-add
//     measured 0-7 % slower), beta = the sum of h's bytes (v_sad_u8), taken as the
//     binary16 number 1024 + beta by placing it in that number's mantissa, two
//     states in one register.  Then
//     d = beta - 510 (exact) and level = fma(d, k_hi, fma(d, k_lo, e)) in
//     binary16 with k_hi + k_lo = 1 / std and e = (510 - mean) / std: equal bit
//     for bit to the table's binary16 rounding for every beta in 0..1020 that
//     the table holds (the tests compare all 65,536 states).  4.75 instructions
//     a weight with the window.
//   mcg, 3INST: w = a s + b mod 2^32 in the same way, masked, and the sum of
//     its two binary16 halves for two states at once.
// Any other table, any within-tile order and K = 5..8 take the general form:
// every element's window by its position, and its level from the table.
#pragma once

#include "exl3_internal.h"

namespace exl3 {

using f16x2 = _Float16 __attribute__((ext_vector_type(2)));
using f16x8 = _Float16 __attribute__((ext_vector_type(8)));
using bf16x2 = __bf16 __attribute__((ext_vector_type(2)));
using bf16x8 = __bf16 __attribute__((ext_vector_type(8)));
using f32x4 = float __attribute__((ext_vector_type(4)));
// with the alignment of their elements
using f32x4u = float __attribute__((ext_vector_type(4), aligned(4)));
using u32x4u = uint32_t __attribute__((ext_vector_type(4), aligned(2)));
using u32x2u = uint32_t __attribute__((ext_vector_type(2), aligned(2)));
using f32x16 = float __attribute__((ext_vector_type(16)));
using u32x4 = uint32_t __attribute__((ext_vector_type(4)));
using u32x2 = uint32_t __attribute__((ext_vector_type(2)));
using i16x4 = short __attribute__((ext_vector_type(4)));

// The wave's number in its workgroup, as a value the compiler knows to be the
// same for all lanes.
__device__ __forceinline__ int wave_number() {
    return __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
}

// How levels are found; the values are template arguments of the kernels.
enum { kLevelsMul1 = 0, kLevelsHalves = 1, kLevelsTable = 2 };

struct Levels {
    uint32_t a, b;           // kLevelsHalves: w = a s + b
    const uint16_t *table;   // kLevelsTable: 65,536 binary16 values
    const uint8_t *inv;      // element -> position within a tile, or null (kLevelsTable only)
    int K;                   // bits a weight (kLevelsTable only; otherwise a template argument)
    float norm;              // a power of two that takes the table's largest level below 4, the
                             // procedural codebooks' range (kLevelsTable only)
};

// The levels of two states as two binary16 values.
template <int LV>
__device__ __forceinline__ uint32_t level_pair(uint32_t s0, uint32_t s1, const Levels &lv) {
    if (LV == kLevelsMul1) {
        const uint32_t h0 = s0 * 0x9E3779B1u, h1 = s1 * 0x9E3779B1u;
        uint32_t p = __builtin_amdgcn_sad_u8(h0, 0u, 0x64006400u);
        p = __builtin_amdgcn_sad_hi_u8(h1, 0u, p);
        const f16x2 base = __builtin_bit_cast(f16x2, 0xE5FEE5FEu);   // -1534
        const f16x2 k_hi = __builtin_bit_cast(f16x2, 0x1EEC1EECu);
        const f16x2 k_lo = __builtin_bit_cast(f16x2, 0x00110011u);
        const f16x2 e = __builtin_bit_cast(f16x2, 0x0C580C58u);
        const f16x2 d = __builtin_bit_cast(f16x2, p) + base;
        const f16x2 c = __builtin_elementwise_fma(d, k_hi, __builtin_elementwise_fma(d, k_lo, e));
        return __builtin_bit_cast(uint32_t, c);
    } else if (LV == kLevelsHalves) {
        const uint32_t w0 = ((s0 * lv.a + lv.b) & 0x8FFF8FFFu) ^ 0x3B603B60u;
        const uint32_t w1 = ((s1 * lv.a + lv.b) & 0x8FFF8FFFu) ^ 0x3B603B60u;
        const f16x2 lo = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(w1, w0, 0x05040100u));
        const f16x2 hi = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(w1, w0, 0x07060302u));
        return __builtin_bit_cast(uint32_t, lo + hi);
    } else {
        return (uint32_t)lv.table[s0] | ((uint32_t)lv.table[s1] << 16);
    }
}

// Words a lane loads for one row of a tile (K = 0: the general form, which
// loads its words when it decodes).
template <int K>
struct RowWords {
    static constexpr int N = K == 0 ? 1 : (K % 2 == 0) ? K / 2 + 1 : (K + 3) / 2;
};

// The words that hold row r's 16 K bits and the 16 bits before them (the
// stream is circular): from word ((K r + 1) >> 1) - 1 on.  For odd K and odd r
// the bits start at that word's first bit and the last word loaded is not
// used (it is held inside the tile); otherwise they start at its 17th bit.
template <int K>
__device__ __forceinline__ void load_row(const uint32_t *tile, int r,
                                         uint32_t (&d)[RowWords<K>::N]) {
    if constexpr (K > 0) {
        const int first = ((K * r + 1) >> 1) - 1;
        d[0] = tile[first < 0 ? 8 * K - 1 : first];
#pragma unroll
        for (int i = 1; i < RowWords<K>::N; ++i) {
            int w = first + i;
            if (K % 2 != 0 && i == RowWords<K>::N - 1) w = w < 8 * K ? w : 8 * K - 1;
            d[i] = tile[w];
        }
    }
}

// The 16 levels of row r of a tile, as the operands of two steps.
template <int LV, int K>
__device__ __forceinline__ void decode_row(const uint32_t *tile, int r,
                                           const uint32_t (&d)[RowWords<K>::N], const Levels &lv,
                                           u32x4 (&out)[2]) {
    if constexpr (K == 0) {
        const int kk = lv.K, nbits = 256 * kk, nc = 8 * kk;
#pragma unroll 2
        for (int j = 0; j < 16; j += 2) {
            uint32_t s[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int el = 16 * r + j + h;
                const int t = lv.inv ? (int)lv.inv[el] : el;
                int p = (t + 1) * kk - 16;
                if (p < 0) p += nbits;
                const int c = p >> 5;
                const uint32_t hi = tile[c], lo = tile[c + 1 == nc ? 0 : c + 1];
                s[h] = __funnelshift_l(lo, hi, (unsigned)(p & 31)) >> 16;
            }
            out[j >> 3][(j >> 1) & 3] = level_pair<kLevelsTable>(s[0], s[1], lv);
        }
    } else {
        // e[q]: the 32 bits that start 16 q bits after the row's run starts
        uint32_t e[K + 1];
        if constexpr (K % 2 == 0) {
#pragma unroll
            for (int q = 0; q <= K; ++q)
                e[q] = (q & 1) ? d[(q + 1) / 2]
                     : q == K  ? d[K / 2] << 16
                               : __builtin_amdgcn_alignbit(d[q / 2], d[q / 2 + 1], 16);
        } else {
            constexpr int NN = (K + 1) / 2;
            uint32_t m[NN];
#pragma unroll
            for (int i = 0; i < NN; ++i)
                m[i] = (r & 1) ? d[i] : __builtin_amdgcn_alignbit(d[i], d[i + 1], 16);
#pragma unroll
            for (int q = 0; q <= K; ++q)
                e[q] = !(q & 1) ? m[q / 2]
                     : q == K   ? m[(K - 1) / 2] << 16
                                : __builtin_amdgcn_alignbit(m[(q - 1) / 2], m[(q + 1) / 2], 16);
        }
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            const int b0 = (j + 1) * K, b1 = (j + 2) * K;
            const uint32_t s0 = (e[b0 >> 4] >> (16 - (b0 & 15))) & 0xFFFFu;
            const uint32_t s1 = (e[b1 >> 4] >> (16 - (b1 & 15))) & 0xFFFFu;
            out[j >> 3][(j >> 1) & 3] = level_pair<LV>(s0, s1, lv);
        }
    }
}

// Binary16 and bfloat16 activations: conversions and the matrix instruction.
template <bool BF>
struct Act;

// The type chosen at run time.
__device__ __forceinline__ float act_load(bool bf, uint16_t v) {
    return bf ? __builtin_bit_cast(float, (uint32_t)v << 16)
              : (float)__builtin_bit_cast(_Float16, v);
}
__device__ __forceinline__ uint16_t act_store(bool bf, float v) {
    return bf ? __builtin_bit_cast(uint16_t, (__bf16)v) : __builtin_bit_cast(uint16_t, (_Float16)v);
}

template <>
struct Act<false> {
    static __device__ __forceinline__ float load(uint16_t v) {
        return (float)__builtin_bit_cast(_Float16, v);
    }
    static __device__ __forceinline__ uint16_t store(float v) {
        return __builtin_bit_cast(uint16_t, (_Float16)v);
    }
    static __device__ __forceinline__ uint32_t store2(float a, float b) {
        f16x2 v;
        v[0] = (_Float16)a;
        v[1] = (_Float16)b;
        return __builtin_bit_cast(uint32_t, v);
    }
    static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
};
template <>
struct Act<true> {
    static __device__ __forceinline__ float load(uint16_t v) {
        return __builtin_bit_cast(float, (uint32_t)v << 16);
    }
    static __device__ __forceinline__ uint16_t store(float v) {
        return __builtin_bit_cast(uint16_t, (__bf16)v);
    }
    static __device__ __forceinline__ uint32_t store2(float a, float b) {
        bf16x2 v;
        v[0] = (__bf16)a;
        v[1] = (__bf16)b;
        return __builtin_bit_cast(uint32_t, v);
    }
    static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
};

// Waits until at most `loads` of the wave's vector loads are under way and its
// shared-memory reads are done (the counts' places in the instruction).
template <int kLoads>
__device__ __forceinline__ void wait_loads() {
    __builtin_amdgcn_s_waitcnt((kLoads & 15) | (7 << 4) | ((kLoads >> 4) << 14));
}

// 16 bytes a lane straight into shared memory, at to + 16 lane.
__device__ __forceinline__ void load_to_lds(const void *from, void *to) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from,
                                     (__attribute__((address_space(3))) void *)to, 16, 0, 0);
}

// Turns 4 x 16 elements of 16 bits: of 16 lanes, lane 4 j + q names elements
// 4 q .. 4 q + 3 of row j, and lane i gets element i of rows 0..3.
__device__ __forceinline__ u32x2 read_turned(const char *from) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) i16x4 *)from));
}

// The workgroup's barrier, across which neither memory accesses nor the
// compiler's schedule move.
__device__ __forceinline__ void barrier_in_place() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// v of lane ^ M, M = 1, 2, 4 or 8, by moves within rows of 16 lanes.
template <int M>
__device__ __forceinline__ float lane_xor(float v) {
    int i = __builtin_bit_cast(int, v);
    if (M == 1) i = __builtin_amdgcn_mov_dpp(i, 0xB1, 0xF, 0xF, true);    // quad 1, 0, 3, 2
    if (M == 2) i = __builtin_amdgcn_mov_dpp(i, 0x4E, 0xF, 0xF, true);    // quad 2, 3, 0, 1
    if (M == 4) {                                                         // ^ 7, then ^ 3
        i = __builtin_amdgcn_mov_dpp(i, 0x141, 0xF, 0xF, true);
        i = __builtin_amdgcn_mov_dpp(i, 0x1B, 0xF, 0xF, true);
    }
    if (M == 8) i = __builtin_amdgcn_mov_dpp(i, 0x128, 0xF, 0xF, true);   // rotation by 8
    return __builtin_bit_cast(float, i);
}

// Natural-order Sylvester Hadamard transform, without its factor, of blocks of
// `had` (64 or 128) consecutive values, eight a lane: three stages in
// registers, three or four across lanes.
template <int M>
__device__ __forceinline__ void hadamard_stage(float (&v)[8]) {
    const float sign = ((threadIdx.x & 63) & M) ? -1.0f : 1.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __builtin_fmaf(v[i], sign, lane_xor<M>(v[i]));
}
__device__ __forceinline__ void hadamard8(float (&v)[8], int had) {
#pragma unroll
    for (int s = 1; s < 8; s <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(i & s)) {
                const float a = v[i], b = v[i + s];
                v[i] = a + b;
                v[i + s] = a - b;
            }
    hadamard_stage<1>(v);
    hadamard_stage<2>(v);
    hadamard_stage<4>(v);
    if (had == 128) hadamard_stage<8>(v);
}

// The power of two that takes a largest magnitude (its bits as an integer) into
// [2^13, 2^14): `scale` its inverse, held in the normal range, and up * up2 the
// power itself, in two factors as it may pass the largest.
struct PowerOfTwo {
    float scale, up, up2;
    bool bad;                 // the largest is NaN or infinite
};
__device__ __forceinline__ PowerOfTwo scale_for(uint32_t big) {
    PowerOfTwo p;
    p.bad = big >= 0x7F800000u;
    // big in [2^(ex - 127), 2^(ex - 126)); its scale 2^(ex - 140)
    int ex = (int)(big >> 23);
    ex = ex < 14 ? 14 : ex;
    p.scale = __builtin_bit_cast(float, (uint32_t)(ex - 13) << 23);
    const int back = 140 - ex;
    p.up = __builtin_bit_cast(float, (uint32_t)(127 + back / 2) << 23);
    p.up2 = __builtin_bit_cast(float, (uint32_t)(127 + back - back / 2) << 23);
    return p;
}

// The group (expert) of a row among `groups` ascending offsets[groups + 1]:
// the number of groups that end at or before it (a row at or past the last
// offset gives `groups`).  All 64 lanes of the wave take part.
__device__ __forceinline__ int group_of_row(const int32_t *offsets, int groups, int64_t row) {
    const int lane = threadIdx.x & 63;
    int e = 0;
    for (int j = 0; j < groups; j += 64) {
        const bool past = j + lane < groups && (int64_t)offsets[1 + j + lane] <= row;
        e += __popcll(__ballot(past));
    }
    return e;
}

// A group's rows [lo, hi), held inside [0, n) whatever the offsets say.
__device__ __forceinline__ void group_rows(const int32_t *offsets, int e, int64_t n, int64_t &lo,
                                           int64_t &hi) {
    lo = 0;
    hi = n;
    if (offsets) {
        lo = offsets[e];
        hi = offsets[e + 1];
        lo = lo < 0 ? 0 : lo;
        hi = hi > n ? n : hi;
    }
}

// Tiles of `per` rows of the groups g0 .. g0 + ng - 1, counted in order of the
// groups (a group's last may be partly empty).  All 64 lanes take part.
__device__ __forceinline__ int tiles_of_group(const int32_t *offsets, int e, bool in, int64_t n,
                                              int per) {
    int64_t a = 0, b = 0;
    if (in) group_rows(offsets, e, n, a, b);
    return b > a ? (int)((b - a + per - 1) / per) : 0;
}

// At most `most`, the grid's: offsets that claim rows over and over could count more
// than an integer holds (each of 65,535 groups up to 2^24 / per).
__device__ __forceinline__ int count_tiles(const int32_t *offsets, int g0, int ng, int64_t n,
                                           int per, int most) {
    const int lane = threadIdx.x & 63;
    int64_t sum = 0;
    for (int j = lane; j < ng + lane; j += 64) sum += tiles_of_group(offsets, g0 + j, j < ng, n, per);
    int some = sum < most ? (int)sum : most;     // 64 of them: most is below 2^25
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) some += __shfl_xor(some, s);
    return some < most ? some : most;
}

// The group that holds tile nt, which becomes the tile's number within it.
__device__ __forceinline__ int group_of_tile(const int32_t *offsets, int g0, int ng, int64_t n,
                                             int per, int &nt) {
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int j = 0; j < ng; j += 64) {
        int sum = tiles_of_group(offsets, g0 + j + lane, j + lane < ng, n, per);
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) {
            const int o = __shfl_up(sum, s);
            if (lane >= s) sum += o;
        }
        const uint64_t past = __ballot(before + sum > nt);
        if (past) {
            const int l = __ffsll((unsigned long long)past) - 1;
            const int prev = l ? __shfl(sum, l - 1) : 0;
            nt -= before + prev;
            return g0 + j + l;
        }
        before += __shfl(sum, 63);
    }
    return -1;
}

// Consecutive workgroups go to different dies: the number of a workgroup's tile
// such that each die takes a run of the `total` tiles.
__device__ __forceinline__ int tile_of_die(int id, int total) {
    const int per = total / 8, rest = total % 8, die = id % 8;
    return die * per + (die < rest ? die : rest) + id / 8;
}

// ---- arguments and launchers of the products (linear.hip, dense.hip, adapters.hip) ----

struct WeightArgs {
    const uint32_t *packed;   // [groups][rows / 16][cols / 16][8 K]
    const float *scale, *su, *sv;
    int groups, rows, cols, K, had;
    int lv_kind;              // kLevels*
    Levels lv;
};

struct AdapterArgs {
    const void *a, *b;        // [count][rank][cols], [count][rows][rank]
    const float *alpha;
    const int32_t *ids;       // [n]
    int count, rank, rank_pad;
    const float *vs;          // [n]: what v's rows are multiplied by (binary16), or null
};

// A launch takes fewer than 2^32 lanes along a grid's side: rows (or pieces) a
// launch, for kernels of `lanes` lanes each.
inline int64_t rows_a_launch(int64_t lanes) {
    const int64_t most = (((int64_t)1 << 31) / lanes);
    return most < 1 ? 1 : most;
}

// x' = H_r (sv x) as binary16 [n][cols] with a scale [n] (a power of two).
hipError_t launch_rotate(const WeightArgs &w, const int32_t *offsets, const void *x, int64_t ldx,
                         int64_t n, bool bf16, uint16_t *xh, float *xs, hipStream_t stream);

// Few rows: part[split][n][rows], sums over a split's columns of x' and the
// levels, from x' and its scales or, where xh is null, from x itself.  With xh null
// and arrived not (run = 1), also y itself; arrived: zero, one count for each group
// and 128 rows of W, zero again afterwards.
struct RowsArgs {
    const uint16_t *xh;
    const float *xs;
    const void *x;
    int64_t ldx;
    bool bf16;
    int64_t n;
    int split, run;           // splits of 2,048 columns; tiles of 16 rows of W a workgroup
    float *part;
    uint32_t *arrived;
    const AdapterArgs *ad;
    const uint16_t *v;
    void *y;
    int64_t ldy;
};
hipError_t launch_coded_rows(const WeightArgs &w, const int32_t *offsets, const RowsArgs &a,
                             hipStream_t stream);

// part[split][n][rows]: sums over a split's columns of x' and the levels, `per`
// (32, 64 or 128) rows of x at a time, staged in shared memory; with split = 1 y
// itself instead.  packed is 16-byte aligned and decoded by formula (lv_kind is
// not kLevelsTable).  transposed: the other direction, where w holds the sizes
// and factors the other way round (rows and su are those of W's columns); packed
// is as it was.
hipError_t launch_coded_tiles(const WeightArgs &w, const int32_t *offsets, const uint16_t *xh,
                              const float *xs, int64_t n, bool transposed, int per, int split,
                              float *part, bool bf16, const AdapterArgs *ad, const uint16_t *v, void *y,
                              int64_t ldy, hipStream_t stream);

// y = su H_l (sum of the parts) scale / had, plus the adapters' products v B^T.
hipError_t launch_finish(const WeightArgs &w, const int32_t *offsets, const float *part, int split,
                         int64_t n, bool bf16, const AdapterArgs *ad, const uint16_t *v, void *y,
                         int64_t ldy, hipStream_t stream);

// The dense weights in the activations' type: [groups][rows][cols], or
// [groups][cols][rows] when transposed; groups g0 .. g0 + ng - 1.  With offsets
// and g0 = 0 also sets the rows of y that no group holds to zero.  Binary16
// weights are divided by powers of two (DenseScale) from inner, launch_inner's.
hipError_t launch_dense(const WeightArgs &w, const int32_t *offsets, int64_t n, int g0, int ng,
                        bool transposed, bool bf16, const int32_t *inner, uint16_t *dense, void *y,
                        int64_t ldy, hipStream_t stream);

// inner[groups]: the exponent of the largest of each group's factors on the side
// that is contracted (sv, or su when transposed).
hipError_t launch_inner(const WeightArgs &w, bool transposed, int32_t *inner, hipStream_t stream);

// What binary16 dense weights were divided by, row by row: 2 to the sum of the
// exponents of scale[g] / div, of out[g][row] and of inner[g] + 1.
struct DenseScale {
    const float *scale, *out;
    const int32_t *inner;
    float div;
};

// y[n][m] = x[n][k] dense[g][m][k]^T for the rows of groups g0 .. g0 + ng - 1,
// plus the adapters' products v b^T (b: [count][m][rank]).  ds: read for binary16.
hipError_t launch_gemm(const void *x, int64_t ldx, const uint16_t *dense, const DenseScale &ds,
                       int64_t n, int m, int k, const int32_t *offsets, int g0, int ng, bool bf16,
                       const AdapterArgs *ad, const void *b, const uint16_t *v, void *y,
                       int64_t ldy, int n_cu, hipStream_t stream);

// Rows of x copied to [n][k] without gaps.
hipError_t launch_pack_rows(const void *x, int64_t ldx, int64_t n, int k, uint16_t *out,
                            hipStream_t stream);

// v[n][rank_pad] = alpha_a x a_a^T in the activations' type, zero past the rank
// and for rows without an adapter; a: [count][rank][k].  vt, if not null, also
// gets v transposed, [rank_pad][ldvt] (rows with an adapter only).  In binary16
// a row of v is stored over a power of two vs[t], and of vt over ts[t], which rows
// of one adapter among 16 share (rows with an adapter only; vs may be null, and
// both are for bfloat16).  One launch takes up to two such products.
struct ShrinkArgs {
    const uint16_t *a, *x;
    int64_t ldx;
    int k;
    uint16_t *v, *vt;
    int64_t ldvt;
    float *vs, *ts;
};
hipError_t launch_shrink(const AdapterArgs &ad, const ShrinkArgs *p, int products, int64_t n,
                         bool bf16, hipStream_t stream);

// [count][p][q] -> [count][q][p], 16-bit elements, up to two arrays.
struct TransposeArgs {
    const uint16_t *src;
    uint16_t *dst;
    int p, q;
};
hipError_t launch_transpose16(const TransposeArgs *t, int arrays, int count, hipStream_t stream);

// out[a][i][j] = sum over the rows t of adapter a of u[t][i] q[t][j], i < rank;
// written as [count][rank][k], or [count][k][rank] when transposed.  ut: u
// transposed, rows 16-byte aligned and ldut >= n rounded up to 32 apart.  part:
// float [splits][count][rank][k].  us: launch_shrink's ts (binary16).  Up to two
// products of equal n and splits.
struct GradArgs {
    const uint16_t *ut, *q;
    const float *us;
    int64_t ldut, ldq;
    int k;
    bool transposed;
    float *part;
    uint16_t *out;
};
// used: [splits][count] bytes, set to whether a split has rows of an adapter (the
// parts of those that have none are not written).
int adapter_grad_splits(int64_t n, int count);
hipError_t launch_adapter_grad(const AdapterArgs &ad, const GradArgs *p, int products, int64_t n,
                               bool bf16, int splits, uint8_t *used, hipStream_t stream);

}  // namespace exl3
