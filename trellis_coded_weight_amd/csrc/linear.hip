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
// A workgroup per row, eight columns a lane at a time, up to kKeep rounds of
// which stay in registers until the row's largest magnitude is known (wider rows
// are transformed a second time).  x' is held in binary16, whose products with
// the levels (binary16 themselves) the matrix instruction sums in binary32.  The
// row's scale is the power of two that takes its largest magnitude into
// [2^13, 2^14): rounding then costs 2^-12 of each value down to 2^-27 of the
// largest, whatever the range of the activations (bfloat16's is far wider than
// binary16's).  A row with a NaN or an infinity becomes NaN throughout.
constexpr int kKeep = 4;

template <bool BF, int THREADS>
__global__ void __launch_bounds__(THREADS)
rotate_kernel(const uint16_t *__restrict__ x, int64_t ldx, int cols, int had, bool wide,
              const float *__restrict__ sv, const int32_t *__restrict__ offsets, int groups,
              uint16_t *__restrict__ xh, float *__restrict__ xs) {
    __shared__ float wave_big[THREADS / 64];
    const int64_t row = blockIdx.x;
    if (offsets) {
        const int e = group_of_row(offsets, groups, row);
        sv += (size_t)(e < groups ? e : groups - 1) * cols;
    }
    const uint16_t *xr = x + row * ldx;
    float v[kKeep][8];
    auto transformed = [&](int col, float (&o)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = 0.0f;
        if (col < cols) {
            uint16_t q[8];
            if (wide) {
                const u32x4 w = *reinterpret_cast<const u32x4 *>(xr + col);
#pragma unroll
                for (int i = 0; i < 8; ++i) q[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) q[i] = xr[col + i];
            }
            const f32x4 s0 = *reinterpret_cast<const f32x4u *>(sv + col);
            const f32x4 s1 = *reinterpret_cast<const f32x4u *>(sv + col + 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = Act<BF>::load(q[i]) * (i < 4 ? s0[i] : s1[i - 4]);
        }
        hadamard_lanes(o, had);
    };
    const int rounds = (cols + THREADS * 8 - 1) / (THREADS * 8);
    // magnitudes compare as integers; NaN and infinity come out on top
    uint32_t big = 0;
    auto largest = [&](const float (&o)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t m = __builtin_bit_cast(uint32_t, o[i]) & 0x7FFFFFFFu;
            big = m > big ? m : big;
        }
    };
#pragma unroll
    for (int c = 0; c < kKeep; ++c)
        if (c < rounds) {
            transformed((c * THREADS + threadIdx.x) * 8, v[c]);
            largest(v[c]);
        }
    for (int c = kKeep; c < rounds; ++c) {
        float o[8];
        transformed((c * THREADS + threadIdx.x) * 8, o);
        largest(o);
    }
    for (int m = 1; m < 64; m <<= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)big, m);
        big = o > big ? o : big;
    }
    if ((threadIdx.x & 63) == 0) wave_big[threadIdx.x >> 6] = __builtin_bit_cast(float, big);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) {
        const uint32_t o = __builtin_bit_cast(uint32_t, wave_big[i]);
        big = o > big ? o : big;
    }
    const bool bad = big >= 0x7F800000u;
    // exponent of the largest: big in [2^(ex - 127), 2^(ex - 126)); its scale
    // 2^(ex - 140), held in the normal range, and the inverse in two factors as
    // it may pass the largest power
    int ex = (int)(big >> 23);
    ex = ex < 14 ? 14 : ex;
    const float scale = __builtin_bit_cast(float, (uint32_t)(ex - 13) << 23);
    const int back = 140 - ex;
    const float up = __builtin_bit_cast(float, (uint32_t)(127 + back / 2) << 23);
    const float up2 = __builtin_bit_cast(float, (uint32_t)(127 + back - back / 2) << 23);
    auto store = [&](int col, const float (&o)[8]) {
        if (col >= cols) return;
        u32x4 out;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t h = Act<false>::store2(o[2 * i] * up * up2, o[2 * i + 1] * up * up2);
            out[i] = bad ? 0x7E007E00u : h;
        }
        *reinterpret_cast<u32x4 *>(xh + row * cols + col) = out;
    };
#pragma unroll
    for (int c = 0; c < kKeep; ++c)
        if (c < rounds) store((c * THREADS + threadIdx.x) * 8, v[c]);
    for (int c = kKeep; c < rounds; ++c) {
        float o[8];
        transformed((c * THREADS + threadIdx.x) * 8, o);
        store((c * THREADS + threadIdx.x) * 8, o);
    }
    if (threadIdx.x == 0) xs[row] = scale;
}

// ---- C x' ----
// A workgroup of eight waves per 16 rows of W, group and split; the waves take
// the split's units of 256 columns in turn, and their sums meet in shared
// memory.  A wave decodes 16 x 64 weights into the operands of two steps and
// uses them for NT tiles of 16 activation rows; x' comes from the caches.
// Columns a wave takes at a time.
constexpr int kUnit = 256;

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
        f32x4 acc[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            int64_t tok = t0 + 16 * t + r;
            tok = tok < hi ? tok : hi - 1;     // a row past the end repeats the last, unstored
            xr[t] = xh + tok * cols;
            acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        for (int u = sp * 8 + wv; u < units; u += 8 * split) {
            const int c0 = u * kUnit;
            uint32_t d[4][RowWords<K>::N];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (c0 + 64 * q < cols)
                    load_row<K>(wrow + (size_t)(c0 / 16 + 4 * q + g) * (8 * kk), r, d[q]);
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
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) sums[wv][t][lane] = acc[t];
        __syncthreads();
        for (int i = threadIdx.x; i < NT * 64; i += 512) {
            const int t = i >> 6, l = i & 63;
            f32x4 a = sums[0][t][l];
#pragma unroll
            for (int w = 1; w < 8; ++w) a += sums[w][t][l];
            const int64_t tok = t0 + 16 * t + (l & 15);
            if (tok < hi)
                *reinterpret_cast<f32x4 *>(part + ((size_t)sp * n + tok) * rows + rt * 16 +
                                           4 * (l >> 4)) = a * xs[tok];
        }
        __syncthreads();
    }
}

// ---- C x' for many rows ----
// A workgroup of four waves per 128 rows of W, 16 NT rows of x' and split of the
// columns.  A step of 64 columns of x' and of the codes' words comes straight
// into one of four places in shared memory (three at K = 4), steps ahead.  A wave decodes
// its 32 x 64 weights of the next step while the matrix instructions multiply
// this step's with the 16 NT rows.  The 32 x 32 x 16 instruction holds the issue
// port for half of its 32 cycles, so about four vector instructions run under
// each (the 16 x 16 x 32 one holds it throughout: the two kinds of work then add
// up, measured).  A lane takes one row of one of two tiles for every 32 columns,
// 16 weights, the operands of two products: columns 16 g + 8 f on, g its half of
// the wave.  Piece s of 16 bytes of row r of x' holds its piece s ^ (r / 2 & 7):
// reads meet no bank twice.
template <int LV, int K, int NT>
__global__ void __launch_bounds__(256, 2)
coded_tiles_kernel(const uint32_t *__restrict__ packed, Levels lv, int rows, int cols,
                   const int32_t *__restrict__ offsets, int groups,
                   const uint16_t *__restrict__ xh, const float *__restrict__ xs, int64_t n,
                   int split, int row_blocks, int total, float *__restrict__ part) {
    constexpr int kRows = 16 * NT, kPieces = kRows * 8 / 256;   // of x', a thread and step
    constexpr int kX = kRows * 128, kPlace = kX + 1024 * K;     // bytes of a place: x', words
    // places: as many as leave two workgroups' worth of shared memory
    constexpr int kRing = 4 * kPlace < 80 * 1024 ? 4 : 3;
    __shared__ __align__(16) char ring[kRing * kPlace];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int r = lane & 31, g = lane >> 5;
    // each die takes a run of tiles: row blocks of W one after the other for the
    // same rows of x'
    if (offsets) {
        const int tiles = count_tiles(offsets, 0, groups, n, kRows) * row_blocks * split;
        total = tiles < total ? tiles : total;
        if ((int)blockIdx.x >= total) return;    // fewer tiles than the grid allows for
    }
    const int id = tile_of_die(blockIdx.x, total), rb = id % row_blocks;
    int nt = id / row_blocks, e = 0;
    const int sp = nt % split;
    nt /= split;
    int64_t lo = 0, hi = n;
    if (offsets) {
        e = group_of_tile(offsets, 0, groups, n, kRows, nt);
        if (e < 0) return;
        group_rows(offsets, e, n, lo, hi);
    }
    const int64_t t0 = lo + (int64_t)nt * kRows;
    const int row_tiles = rows / 16, all = cols / 64;
    const int first = (int)((int64_t)all * sp / split);
    const int steps = (int)((int64_t)all * (sp + 1) / split) - first;

    // x': pieces from a uniform base that moves along the columns
    const char *x_at = reinterpret_cast<const char *>(xh + t0 * cols + (size_t)first * 64);
    uint32_t piece_at[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const int q = i * 256 + threadIdx.x, row = q >> 3;
        const int64_t left = hi - t0 - 1;    // past the end: repeats, not stored
        piece_at[i] = (uint32_t)(row < left ? row : left) * (uint32_t)(cols * 2) +
                      ((q & 7) ^ ((row >> 1) & 7)) * 16;
    }
    // words: 8 K pieces of 16 bytes a row tile and step, K loads of 64 lanes,
    // one by each of the first K waves (the others repeat the last one's, so that
    // every wave has as many loads under way)
    const int word_wave = wv < K ? wv : K - 1;
    const int wq = word_wave * 64 + lane;
    int w_tile = rb * 8 + wq / (8 * K);
    w_tile = w_tile < row_tiles ? w_tile : row_tiles - 1;
    const char *w_at = reinterpret_cast<const char *>(packed) +
                       (((size_t)e * row_tiles + w_tile) * (cols / 16) + (size_t)first * 4) * (32 * K) +
                       wq % (8 * K) * 16;
    int loaded = 0, fill = 0;
    auto load = [&]() {
        char *to = ring + fill * kPlace;
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            load_to_lds(x_at + piece_at[i], to + (i * 256 + wv * 64) * 16);
        load_to_lds(w_at, to + kX + word_wave * 1024);
        ++loaded;
        fill = fill + 1 < kRing ? fill + 1 : 0;
        // past the last step: repeats it, into a place that nobody reads
        x_at += loaded < steps ? 128 : 0;
        w_at += loaded < steps ? 128 * K : 0;
    };
    // what a wave needs of a step: its rows' words (then their levels) and the
    // rows of x', for two times 32 columns
    constexpr int NJ = NT / 2;
    struct Operands {
        uint32_t d[2][RowWords<K>::N];
        u32x4 w[2][2], b[NJ][2][2];
    };
    int piece[2][2];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int f = 0; f < 2; ++f)
            piece[c][f] = r * 128 + ((4 * c + 2 * g + f) ^ ((r >> 1) & 7)) * 16;
    const int words_at = kX + ((2 * wv + (r >> 4)) * 4 + g) * (32 * K);
    auto read = [&](int place, Operands &o) {
        const char *at = ring + place * kPlace;
#pragma unroll
        for (int c = 0; c < 2; ++c)
            load_row<K>(reinterpret_cast<const uint32_t *>(at + words_at + 2 * c * 32 * K), r & 15,
                        o.d[c]);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int f = 0; f < 2; ++f)
                    o.b[j][c][f] = *reinterpret_cast<const u32x4 *>(at + j * 4096 + piece[c][f]);
    };
    auto decode = [&](Operands &o) {
#pragma unroll
        for (int c = 0; c < 2; ++c) decode_row<LV, K>(nullptr, r & 15, o.d[c], lv, o.w[c]);
    };
    f32x16 acc[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[j][i] = 0.0f;
    Operands even, odd;
    int here = 0;
    auto step = [&](Operands &cur, Operands &next) {
        // the next step has landed when only the loads of those after it are under way
        __builtin_amdgcn_sched_barrier(0);
        wait_loads<(kRing - 3) * (kPieces + 1)>();
        barrier_in_place();
        __builtin_amdgcn_sched_barrier(0);
        // the next step's reads first: they finish under this step's decoding and
        // products, which alternate
        here = here + 1 < kRing ? here + 1 : 0;
        read(here, next);
        load();                              // over the step before this one
        __builtin_amdgcn_sched_barrier(0);
        decode(next);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                        __builtin_bit_cast(f16x8, cur.w[c][f]),
                        __builtin_bit_cast(f16x8, cur.b[j][c][f]), acc[j], 0, 0, 0);
        // the first products cover the reads' latency
        __builtin_amdgcn_sched_group_barrier(0x8, 2, 0);
#pragma unroll
        for (int q = 0; q < 4 * NJ - 2; ++q) {
            __builtin_amdgcn_sched_group_barrier(0x2, 12, 0);
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        }
    };
    if (steps > 0) {
#pragma unroll
        for (int i = 0; i < kRing - 1; ++i) load();
        wait_loads<(kRing - 2) * (kPieces + 1)>();
        barrier_in_place();
        read(0, even);
        decode(even);
        int s = 0;
        for (; s + 1 < steps; s += 2) {
            step(even, odd);
            step(odd, even);
        }
        if (s < steps) step(even, odd);
    }
    // column (row of x') 32 j + r, rows 8 q + 4 g .. of the wave's 32
    const int row0 = rb * 128 + wv * 32 + 4 * g;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int64_t tok = t0 + 32 * j + r;
        if (tok >= hi) continue;
        const float s = xs[tok];
        float *o = part + ((size_t)sp * n + tok) * rows + row0;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (row0 + 8 * q < rows)
                *reinterpret_cast<f32x4 *>(o + 8 * q) =
                    f32x4{acc[j][4 * q], acc[j][4 * q + 1], acc[j][4 * q + 2],
                          acc[j][4 * q + 3]} * s;
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
    const uint16_t *xx = static_cast<const uint16_t *>(x);
    const bool wide = reinterpret_cast<uintptr_t>(x) % 16 == 0 && ldx % 8 == 0;
#define EXL3_ROTATE(BF, THREADS)                                                               \
    hipLaunchKernelGGL((rotate_kernel<BF, THREADS>), dim3((unsigned)n), dim3(THREADS), 0, stream, \
                       xx, ldx, w.cols, w.had, wide, w.sv, offsets, w.groups, xh, xs)
    // a round a row while that takes at most 512 lanes
    if (bf16 && w.cols <= 2048)
        EXL3_ROTATE(true, 256);
    else if (bf16)
        EXL3_ROTATE(true, 512);
    else if (w.cols <= 2048)
        EXL3_ROTATE(false, 256);
    else
        EXL3_ROTATE(false, 512);
#undef EXL3_ROTATE
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

hipError_t launch_coded_tiles(const WeightArgs &w, const int32_t *offsets, const uint16_t *xh,
                              const float *xs, int64_t n, int split, float *part,
                              hipStream_t stream) {
    constexpr int NT = 8;
    const int row_blocks = (w.rows + 127) / 128;
    const int64_t n_tiles = offsets ? n / (16 * NT) + w.groups : (n + 16 * NT - 1) / (16 * NT);
    const int total = (int)(n_tiles * row_blocks * split);
#define EXL3_TILES(LV, KK)                                                                      \
    case KK:                                                                                    \
        hipLaunchKernelGGL((coded_tiles_kernel<LV, KK, NT>), dim3((unsigned)total), dim3(256),  \
                           0, stream, w.packed, w.lv, w.rows, w.cols, offsets, w.groups, xh, xs, \
                           n, split, row_blocks, total, part);                                  \
        break
    if (w.lv_kind == kLevelsMul1)
        switch (w.K) {
            EXL3_TILES(kLevelsMul1, 1);
            EXL3_TILES(kLevelsMul1, 2);
            EXL3_TILES(kLevelsMul1, 3);
            EXL3_TILES(kLevelsMul1, 4);
            default: return hipErrorInvalidValue;
        }
    else if (w.lv_kind == kLevelsHalves)
        switch (w.K) {
            EXL3_TILES(kLevelsHalves, 1);
            EXL3_TILES(kLevelsHalves, 2);
            EXL3_TILES(kLevelsHalves, 3);
            EXL3_TILES(kLevelsHalves, 4);
            default: return hipErrorInvalidValue;
        }
    else
        return hipErrorInvalidValue;
#undef EXL3_TILES
    return hipGetLastError();
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
