// Products of few and of medium numbers of rows with coded weights, y = x W^T,
// and of the latter y = x W with both sides' transforms and factors exchanged, on
// gfx950.
//
// W = diag(su) H_l (scale C) H_r diag(sv) with C the codes' levels, so
//   y = scale / had * su (H_l (C x')),   x' = H_r (sv x)
// (H here without its factor 1 / sqrt(had), which enters twice).  x' comes from
// rotate_kernel, C x' from the codes in coded_rows_kernel or, for more rows, in
// coded_tiles_kernel.  The left transform and the factors are finish_kernel's; the
// smallest calls take them in coded_rows_kernel, and those whose columns are not
// split in coded_tiles_kernel.
#include "coded.h"

namespace exl3 {

namespace {

// ---- x' ----
// A workgroup per row, eight columns a lane at a time, up to kKeep rounds of
// which stay in registers until the row's largest magnitude is known (wider rows
// are transformed a second time).  x' is held in binary16, whose products with
// the levels (binary16 themselves) the matrix instruction sums in binary32.  The
// row's scale is the power of two that takes its largest magnitude into
// [2^13, 2^14): rounding then costs at most 2^-11 of each value down to 2^-27 of
// the largest, whatever the range of the activations (bfloat16's is far wider than
// binary16's).  A row with a NaN or an infinity becomes NaN throughout.  8,200
// rows of 2,048 columns: 16 us, 4.2 TB/s of both sides, near a copy's 4.7.
constexpr int kKeep = 4;

template <bool BF, int THREADS>
__global__ void __launch_bounds__(THREADS)
rotate_kernel(const uint16_t *__restrict__ x, int64_t ldx, int cols, int had,
              const float *__restrict__ sv, const int32_t *__restrict__ offsets, int groups,
              int64_t row0, uint16_t *__restrict__ xh, float *__restrict__ xs) {
    __shared__ float wave_big[THREADS / 64];
    const int64_t row = row0 + blockIdx.x;
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
            const u32x4 w = *reinterpret_cast<const u32x4u *>(xr + col);
            uint16_t q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
            const f32x4 s0 = *reinterpret_cast<const f32x4u *>(sv + col);
            const f32x4 s1 = *reinterpret_cast<const f32x4u *>(sv + col + 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = Act<BF>::load(q[i]) * (i < 4 ? s0[i] : s1[i - 4]);
        }
        hadamard8(o, had);
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
    const PowerOfTwo p2 = scale_for(big);
    auto store = [&](int col, const float (&o)[8]) {
        if (col >= cols) return;
        u32x4 out;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t h = Act<false>::store2(o[2 * i] * p2.up * p2.up2,
                                                  o[2 * i + 1] * p2.up * p2.up2);
            out[i] = p2.bad ? 0x7E007E00u : h;
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
    if (threadIdx.x == 0) xs[row] = p2.scale;
}

// Eight columns of a row of y, row .. row + 7 of W, from their left transform:
// the factors, the adapter's product v b^T, one rounding.  AHEAD: 16 ranks' loads
// at once, where there are registers.
template <bool AHEAD>
__device__ __forceinline__ void finish_row(float (&z)[8], float f, const float *su,
                                           const AdapterArgs &ad, const uint16_t *v, int id,
                                           int64_t tok, int row, int rows, bool bf16,
                                           uint16_t *y) {
    const f32x4 s0 = *reinterpret_cast<const f32x4u *>(su);
    const f32x4 s1 = *reinterpret_cast<const f32x4u *>(su + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] *= f * (i < 4 ? s0[i] : s1[i - 4]);
    if (v) {
        if (id >= 0 && id < ad.count) {
            const uint16_t *b = static_cast<const uint16_t *>(ad.b) +
                                ((size_t)id * rows + row) * ad.rank;
            const uint16_t *vt = v + tok * ad.rank_pad;
            const float vs = ad.vs ? ad.vs[tok] : 1.0f;
            int k = 0;
            for (; AHEAD && k + 16 <= ad.rank; k += 16) {
                u32x4 vk[2], bk[8][2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    vk[h] = *reinterpret_cast<const u32x4 *>(vt + k + 8 * h);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        bk[i][h] = *reinterpret_cast<const u32x4u *>(b + (size_t)i * ad.rank + k +
                                                                     8 * h);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const float vf =
                            act_load(bf16, (uint16_t)(vk[h][c >> 1] >> (16 * (c & 1)))) * vs;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            z[i] += vf * act_load(bf16, (uint16_t)(bk[i][h][c >> 1] >>
                                                                   (16 * (c & 1))));
                    }
            }
            for (; k < ad.rank; k += 8) {
                const u32x4 vk = *reinterpret_cast<const u32x4 *>(vt + k);
                float vf[8];
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    vf[c] = act_load(bf16, (uint16_t)(vk[c >> 1] >> (16 * (c & 1)))) * vs;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint16_t *bi = b + (size_t)i * ad.rank + k;
                    if (k + 8 <= ad.rank) {
                        const u32x4 bk = *reinterpret_cast<const u32x4u *>(bi);
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            z[i] += vf[c] * act_load(bf16, (uint16_t)(bk[c >> 1] >> (16 * (c & 1))));
                    } else {
                        for (int c = 0; c < 8 && k + c < ad.rank; ++c)
                            z[i] += vf[c] * act_load(bf16, bi[c]);
                    }
                }
            }
        }
    }
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = bf16 ? Act<true>::store2(z[2 * i], z[2 * i + 1])
                    : Act<false>::store2(z[2 * i], z[2 * i + 1]);
    *reinterpret_cast<u32x4u *>(y) = u32x4u{o[0], o[1], o[2], o[3]};
}

// ---- few rows ----
// A workgroup of eight waves takes `run` tiles of 16 rows of W in turn, for one
// group and split.  A split is eight units of 256 columns, and each wave has one
// of them throughout: the operands of x' (16 rows of activations) stay in its
// registers, the words of the next tile are under way while it decodes and
// multiplies this one's, and the eight waves' sums meet in shared memory, in two
// places by turns (one barrier a tile).  Decoding bounds it: 4.75 vector
// instructions a weight and 4.4 cycles each, 7.3 us for the 50 M weights of
// 12288 x 4096 at 1,024 SIMDs and 2.2 GHz, beside reading the codes: 15 us at
// K = 4.
//
// x' comes from rotate_kernel, or (OWN, up to kOwn rows at a time) each wave
// transforms its own unit of x, with a scale for the unit.
//
// The left transform mixes 128 rows of W, eight tiles' sums.  It is left to
// finish_kernel, but for the smallest calls (FINISH, run = 1): there each
// workgroup stores its sums past its die's cache, waits until they are there,
// and counts itself, and the last of a block reads all sums, in the order of the
// splits, and finishes the rows of y.  One launch in place of three: 8.3 us
// for one row and 1024 x 4096 (three took 15.3).  With more workgroups than compute
// units a launch of its own costs less than one tile a workgroup, its stores past the
// die's cache and the late finish do: 12288 x 4096, K = 4, in one launch 23.7 us, in
// two 15.6; 64 rows of 64 experts of 1408 x 2048 51 and 33.
constexpr int kUnit = 256, kOwn = 8;
constexpr int kOwnPitch = kUnit * 2 + 16;        // bytes of a row of a wave's own x'

template <int LV, int K, bool OWN, bool FINISH>
__global__ void __launch_bounds__(512, 4)     // two workgroups a compute unit
coded_rows_kernel(const uint32_t *__restrict__ packed, Levels lv, int rows, int cols, int Kr,
                  int had, const float *__restrict__ scale, const float *__restrict__ su,
                  const float *__restrict__ sv, const int32_t *__restrict__ offsets, int groups,
                  RowsArgs a, AdapterArgs ad) {
    constexpr int kStep = OWN ? kOwn : 16;
    __shared__ f32x4 sums[2][8][64];
    __shared__ __align__(16) char own[OWN ? 8 * kOwn * kOwnPitch : 16];
    __shared__ uint32_t before;
    const int lane = threadIdx.x & 63, wv = wave_number();
    const int r = lane & 15, g = lane >> 4;
    const int row_tiles = rows / 16, runs = (row_tiles + a.run - 1) / a.run;
    const int rt0 = blockIdx.x % runs * a.run, sp = blockIdx.x / runs, e = blockIdx.y;
    const int rt1 = rt0 + a.run < row_tiles ? rt0 + a.run : row_tiles;
    const int64_t n = a.n;
    uint16_t *y = static_cast<uint16_t *>(a.y);
    if (FINISH && offsets) {
        // rows of no group, by all workgroups
        const int64_t from = offsets[0], to = offsets[groups];
        const int64_t all = (int64_t)gridDim.x * gridDim.y;
        const int64_t me = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
        for (int64_t t = me; t < n && t < from; t += all)
            for (int c = threadIdx.x; c < rows; c += 512) y[t * a.ldy + c] = 0;
        for (int64_t t = (to > 0 ? to : 0) + me; t < n; t += all)
            for (int c = threadIdx.x; c < rows; c += 512) y[t * a.ldy + c] = 0;
    }
    int64_t lo, hi;
    group_rows(offsets, e, n, lo, hi);
    if (lo >= hi) return;
    const int kk = K ? K : Kr;
    const int c0 = (sp * 8 + wv) * kUnit;        // the wave's columns; past the last: none
    const int quads = c0 >= cols ? 0 : cols - c0 >= kUnit ? 4 : (cols - c0) / 64;
    const uint32_t *wcol = packed + ((size_t)e * row_tiles * (cols / 16) + c0 / 16 + g) * (8 * kk);
    const size_t wrow = (size_t)(cols / 16) * (8 * kk);
    using Words = uint32_t[4][RowWords<K>::N];
    auto load_tile = [&](int rt, Words &d) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (q < quads) load_row<K>(wcol + rt * wrow + q * 32 * kk, r, d[q]);
    };
    for (int64_t t0 = lo; t0 < hi; t0 += kStep) {
        Words even, odd;
        load_tile(rt0, even);
        u32x4 x[4][2];
        float x_scale = 0.0f;                    // of the lane's row of x'
        if (OWN) {
            char *mine = own + wv * kOwn * kOwnPitch;
            const int here = hi - t0 < kOwn ? (int)(hi - t0) : kOwn;
            // two rows at a time, half a wave each, eight columns a lane
            const int col = c0 + (lane & 31) * 8;
            const bool in = col < cols;
            f32x4 s0 = {0.0f, 0.0f, 0.0f, 0.0f}, s1 = s0;
            if (in) {
                const float *svp = sv + (size_t)e * cols + col;
                s0 = *reinterpret_cast<const f32x4u *>(svp);
                s1 = *reinterpret_cast<const f32x4u *>(svp + 4);
            }
            for (int t = 0; t < here; t += 2) {
                const int row = t + (lane >> 5);
                float o[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
                if (in && row < here) {
                    const uint16_t *xp = static_cast<const uint16_t *>(a.x) +
                                         (t0 + row) * a.ldx + col;
                    const u32x4 w = *reinterpret_cast<const u32x4u *>(xp);
                    uint16_t q[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) q[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        o[i] = act_load(a.bf16, q[i]) * (i < 4 ? s0[i] : s1[i - 4]);
                }
                hadamard8(o, had);
                // magnitudes compare as integers; NaN and infinity come out on top
                uint32_t big = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t m = __builtin_bit_cast(uint32_t, o[i]) & 0x7FFFFFFFu;
                    big = m > big ? m : big;
                }
#pragma unroll
                for (int m = 1; m < 32; m <<= 1) {
                    const uint32_t q = (uint32_t)__shfl_xor((int)big, m);
                    big = q > big ? q : big;
                }
                const PowerOfTwo p2 = scale_for(big);
                u32x4 h;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    h[i] = Act<false>::store2(o[2 * i] * p2.up * p2.up2,
                                              o[2 * i + 1] * p2.up * p2.up2);
                    if (p2.bad) h[i] = 0x7E007E00u;
                }
                if (row < here)
                    *reinterpret_cast<u32x4 *>(mine + row * kOwnPitch + (lane & 31) * 16) = h;
                const float first = __shfl(p2.scale, 0), second = __shfl(p2.scale, 32);
                if (r == t) x_scale = first;
                if (r == t + 1) x_scale = second;
            }
            // the wave's own stores, read back by other lanes of the same wave
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const u32x4 *xp = reinterpret_cast<const u32x4 *>(
                    mine + (r < here ? r : here - 1) * kOwnPitch + q * 128 + g * 32);
                x[q][0] = xp[0];
                x[q][1] = xp[1];
            }
            // these reads are done before the next rows' stores
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        } else {
            int64_t tok = t0 + r;
            tok = tok < hi ? tok : hi - 1;       // past the end: repeats, not stored
            x_scale = a.xs[tok];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (q < quads) {
                    const u32x4 *xp = reinterpret_cast<const u32x4 *>(a.xh + tok * cols + c0 +
                                                                      64 * q + 16 * g);
                    x[q][0] = xp[0];
                    x[q][1] = xp[1];
                }
        }
        auto one_tile = [&](int rt, Words &now, Words &next) {
            f32x4 acc[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
            if (rt + 1 < rt1) load_tile(rt + 1, next);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (q >= quads) break;
                u32x4 w[2];
                decode_row<LV, K>(wcol + rt * wrow + q * 32 * kk, r, now[q], lv, w);
                acc[0] = Act<false>::mfma(w[0], x[q][0], acc[0]);
                acc[1] = Act<false>::mfma(w[1], x[q][1], acc[1]);
            }
            const int place = rt & 1;
            sums[place][wv][lane] = (acc[0] + acc[1]) * x_scale;
            __syncthreads();
            if (wv == (rt & 7)) {
                f32x4 z = sums[place][0][lane];
#pragma unroll
                for (int w = 1; w < 8; ++w) z += sums[place][w][lane];
                const int64_t tok = t0 + r;
                if (tok < hi && r < kStep) {
                    float *o = a.part + ((size_t)sp * n + tok) * rows + rt * 16 + 4 * g;
                    if (FINISH) {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            __hip_atomic_store(o + c, z[c], __ATOMIC_RELAXED,
                                               __HIP_MEMORY_SCOPE_AGENT);
                    } else {
                        *reinterpret_cast<f32x4 *>(o) = z;
                    }
                }
            }
        };
        for (int rt = rt0; rt < rt1; rt += 2) {
            one_tile(rt, even, odd);
            if (rt + 1 < rt1) one_tile(rt + 1, odd, even);
        }
        // the next rows' sums may meet in the place that was just read
        if (t0 + kStep < hi) __syncthreads();
    }
    if (!FINISH) return;
    // count this workgroup once its sums are stored (each wave waits for its own:
    // stores and loads of device scope go past the die's cache, so the count
    // needs to order nothing else)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    const int rb = rt0 / 8, row_blocks = (row_tiles + 7) / 8;
    uint32_t *count = a.arrived + (size_t)e * row_blocks + rb;
    if (threadIdx.x == 0)
        before = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    const int of_block = row_tiles - 8 * rb < 8 ? row_tiles - 8 * rb : 8;
    if (before != (uint32_t)(of_block * a.split) - 1u) return;
    if (threadIdx.x == 0)
        __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    // 16 lanes a row of y, eight of the block's 128 columns a lane
    const int row = rb * 128 + r * 8;
    const bool in = row < rows;
    const float f = scale[e] / (float)had;
    for (int64_t tok0 = lo + wv * 4; tok0 < hi; tok0 += 32) {
        const int64_t tok = tok0 + g;
        float z[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        const bool has = in && tok < hi;
        const int id = has && a.v ? ad.ids[tok] : -1;
        if (has)
            for (int s = 0; s < a.split; ++s) {
                const float *p = a.part + ((size_t)s * n + tok) * rows + row;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    z[i] += __hip_atomic_load(p + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
        hadamard8(z, had);
        if (has)
            finish_row<false>(z, f, su + (size_t)e * rows + row, ad, a.v, id, tok, row, rows,
                              a.bf16, y + tok * a.ldy + row);
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
// reads meet no bank twice.  Decoding and the products share the issue port, which
// bounds it: 8,200 rows of 64 experts, 1408 x 2048, K = 3: 107 us, vector
// instructions for 49 % of the cycles and the matrix units for 26 %; 333 rows,
// 4096 x 4096: 28 us.
// What the kernel needs to finish y itself (y null: it stores sums).
struct TilesOut {
    const float *scale, *su;
    int had;
    AdapterArgs ad;
    const uint16_t *v;
    bool bf16;
    uint16_t *y;
    int64_t ldy;
};

// The other direction, x C (T; rows and cols are then C's columns and rows): a
// lane's 16 levels belong to 16 columns of the result, so the 16 lanes of a tile
// hand them over as they are decoded, through 512 bytes of shared memory and the
// reads that turn 4 x 16 elements; piece h of a row is at h ^ (row / 8), so that
// neither side meets a bank twice.  4,001 rows of 16 experts, 2048 x 1408: 59 us;
// writing the dense weights first took 11 us more for the whole call.
template <int LV, int K, int NT, bool T>
__global__ void __launch_bounds__(256, NT == 8 || (T && K == 4) ? 2 : NT == 4 || T ? 3 : 4)
coded_tiles_kernel(const uint32_t *__restrict__ packed, Levels lv, int rows, int cols,
                   const int32_t *__restrict__ offsets, int groups,
                   const uint16_t *__restrict__ xh, const float *__restrict__ xs, int64_t n,
                   int split, int row_blocks, int total, float *__restrict__ part, TilesOut out) {
    constexpr int kRows = 16 * NT, kPieces = kRows * 8 / 256;   // of x', a thread and step
    constexpr int kX = kRows * 128, kPlace = kX + 1024 * K;     // bytes of a place: x', words
    // places: as many as leave room for two workgroups
    constexpr int kTurn = T ? 4 * 2048 : 0;                     // 2 KiB a wave
    constexpr int kRing = 4 * kPlace + kTurn < 80 * 1024 ? 4 : 3;
    __shared__ __align__(16) char ring[kRing * kPlace + kTurn];
    const int lane = threadIdx.x & 63, wv = wave_number();
    const int r = lane & 31, g = lane >> 5;
    if (offsets && out.y) {
        // rows of no group, by all workgroups
        const int64_t from = offsets[0], to = offsets[groups];
        for (int64_t t = blockIdx.x; t < n && t < from; t += gridDim.x)
            for (int c = threadIdx.x; c < rows; c += 256) out.y[t * out.ldy + c] = 0;
        for (int64_t t = (to > 0 ? to : 0) + blockIdx.x; t < n; t += gridDim.x)
            for (int c = threadIdx.x; c < rows; c += 256) out.y[t * out.ldy + c] = 0;
    }
    // each die takes a run of tiles: row blocks of W one after the other for the
    // same rows of x'
    if (offsets) {
        const int each = row_blocks * split;
        total = count_tiles(offsets, 0, groups, n, kRows, total / each) * each;
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
    const char *w_at = reinterpret_cast<const char *>(packed);
    if (T)
        w_at += (((size_t)e * (cols / 16) + first * 4 + wq % (8 * K) / (2 * K)) * row_tiles + w_tile) *
                    (32 * K) + wq % (2 * K) * 16;
    else
        w_at += (((size_t)e * row_tiles + w_tile) * (cols / 16) + (size_t)first * 4) * (32 * K) +
                wq % (8 * K) * 16;
    const size_t w_step = (size_t)(T ? row_tiles : 1) * (128 * K);
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
        w_at += loaded < steps ? w_step : 0;
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
        for (int c = 0; c < 2; ++c) {
            decode_row<LV, K>(nullptr, r & 15, o.d[c], lv, o.w[c]);
            if constexpr (T) {
                // (a wave's accesses of shared memory are done in their order)
                char *tile = ring + kRing * kPlace + wv * 2048 + (lane >> 4) * 512;
                const int row = lane & 15, q = lane & 3;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *reinterpret_cast<u32x4 *>(tile + row * 32 + (h ^ (row >> 3)) * 16) = o.w[c][h];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const u32x2 v = read_turned(tile + (4 * j + (row >> 2)) * 32 +
                                                ((q >> 1) ^ (j >> 1)) * 16 + 8 * (q & 1));
                    o.w[c][j >> 1][2 * (j & 1)] = v[0];
                    o.w[c][j >> 1][2 * (j & 1) + 1] = v[1];
                }
            }
        }
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
    if (out.y) {
        // The left transform over the 128 rows and the factors, 64 rows of x' at a
        // time.  A lane holds rows 8 q + 4 g + i of its wave's 32: the stages over i
        // and q are in registers; those over g and the waves after shared memory,
        // where a thread takes rows 8 p .. 8 p + 7 of every 32 of one row of x'.
        constexpr int kPitch = 132;              // floats a row of x'
        static_assert((kRows < 64 ? kRows : 64) * kPitch * 4 <= kRing * kPlace, "the sums fit");
        float *sums = reinterpret_cast<float *>(ring);
        wait_loads<0>();
        barrier_in_place();
        const float f = out.scale[e] / (float)out.had;
        const float *su = out.su + (size_t)e * rows + rb * 128;
#pragma unroll
        for (int j0 = 0; j0 < NJ; j0 += 2) {
            if (j0) __syncthreads();             // the last 64 have been read
#pragma unroll
            for (int j = j0; j < j0 + 2 && j < NJ; ++j) {
                f32x16 z = acc[j];
#pragma unroll
                for (int s = 1; s < 16; s <<= 1)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (!(i & s)) {
                            const float a = z[i], b = z[i + s];
                            z[i] = a + b;
                            z[i + s] = a - b;
                        }
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<f32x4 *>(sums + (32 * (j - j0) + r) * kPitch + 32 * wv + 8 * q +
                                               4 * g) =
                        f32x4{z[4 * q], z[4 * q + 1], z[4 * q + 2], z[4 * q + 3]};
            }
            __syncthreads();
            const int t = threadIdx.x >> 2, p = threadIdx.x & 3;
            const int64_t tok = t0 + 32 * j0 + t;
            if (tok >= hi || 32 * j0 + t >= kRows) continue;
            float z[4][8];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const f32x4 *at = reinterpret_cast<const f32x4 *>(sums + t * kPitch + 32 * w + 8 * p);
                const f32x4 a = at[0], b = at[1];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    z[w][i] = a[i] + b[i];
                    z[w][i + 4] = a[i] - b[i];
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float a = z[0][i] + z[1][i], b = z[0][i] - z[1][i];
                const float c = z[2][i] + z[3][i], d = z[2][i] - z[3][i];
                const bool whole = out.had == 128;
                z[0][i] = whole ? a + c : a;
                z[1][i] = whole ? b + d : b;
                z[2][i] = whole ? a - c : c;
                z[3][i] = whole ? b - d : d;
            }
            const float ft = f * xs[tok];
            const int id = out.v ? out.ad.ids[tok] : -1;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int row = 32 * w + 8 * p;
                if (rb * 128 + row < rows)
                    finish_row<false>(z[w], ft, su + row, out.ad, out.v, id, tok, rb * 128 + row,
                                      rows, out.bf16, out.y + tok * out.ldy + rb * 128 + row);
            }
        }
        return;
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
// A wave per row of y and 512 of its columns, eight a lane, in a workgroup of its
// own: the waves of the smaller calls then spread over the compute units (32 x
// 4096 with adapters: 9.4 us with four waves a workgroup, 7.5 with one, 6 with 16
// ranks' loads at once).  Latency
// bounds it: 4 us from the first load to the last store at 24 x 4096, 6.5 at
// 333 x 4096.
__global__ void __launch_bounds__(64)
finish_kernel(const float *__restrict__ part, int split, int64_t n, int rows, int had,
              const float *__restrict__ scale, const float *__restrict__ su,
              const int32_t *__restrict__ offsets, int groups, AdapterArgs ad,
              const uint16_t *__restrict__ v, bool bf16, int64_t tok0, uint16_t *__restrict__ y,
              int64_t ldy) {
    const int lane = threadIdx.x & 63, blocks = (rows + 511) / 512;
    const int here = blockIdx.x / blocks;
    const int64_t tok = tok0 + here;
    const int row = (int)(blockIdx.x - here * blocks) * 512 + lane * 8;
    const bool in = row < rows;
    const int id = v ? ad.ids[tok] : -1;
    int e = 0;
    if (offsets) {
        e = group_of_row(offsets, groups, tok);
        if (e >= groups || tok < offsets[0]) {
            if (in)
                for (int i = 0; i < 8; ++i) y[tok * ldy + row + i] = 0;
            return;
        }
    }
    float z[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (in) {
        // eight splits' loads under way at a time
        const float *at = part + tok * rows + row;
        const size_t pitch = (size_t)n * rows;
        for (int s0 = 0; s0 < split; s0 += 8) {
            f32x4 p[8][2];
#pragma unroll
            for (int s = 0; s < 8; ++s)
                if (s0 + s < split) {
                    const f32x4 *q = reinterpret_cast<const f32x4 *>(at + (s0 + s) * pitch);
                    p[s][0] = q[0];
                    p[s][1] = q[1];
                }
#pragma unroll
            for (int s = 0; s < 8; ++s)
                if (s0 + s < split)
#pragma unroll
                    for (int i = 0; i < 8; ++i) z[i] += p[s][i >> 2][i & 3];
        }
    }
    hadamard8(z, had);
    if (in)
        finish_row<true>(z, scale[e] / (float)had, su + (size_t)e * rows + row, ad, v, id, tok, row,
                         rows, bf16, y + tok * ldy + row);
}

template <int LV, int K>
hipError_t coded_rows_t(const WeightArgs &w, const int32_t *offsets, const RowsArgs &a,
                        hipStream_t stream) {
    const int runs = (w.rows / 16 + a.run - 1) / a.run;
    const dim3 grid((unsigned)(runs * a.split), (unsigned)w.groups);
    const AdapterArgs ad = a.ad ? *a.ad : AdapterArgs{};
#define EXL3_ROWS(OWN, FINISH)                                                               \
    hipLaunchKernelGGL((coded_rows_kernel<LV, K, OWN, FINISH>), grid, dim3(512), 0, stream,  \
                       w.packed, w.lv, w.rows, w.cols, w.K, w.had, w.scale, w.su, w.sv,      \
                       offsets, w.groups, a, ad)
    if (a.xh)
        EXL3_ROWS(false, false);
    else if (a.arrived)
        EXL3_ROWS(true, true);
    else
        EXL3_ROWS(true, false);
#undef EXL3_ROWS
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rotate(const WeightArgs &w, const int32_t *offsets, const void *x, int64_t ldx,
                         int64_t n, bool bf16, uint16_t *xh, float *xs, hipStream_t stream) {
    const uint16_t *xx = static_cast<const uint16_t *>(x);
#define EXL3_ROTATE(BF, THREADS)                                                              \
    hipLaunchKernelGGL((rotate_kernel<BF, THREADS>), dim3(rows), dim3(THREADS), 0, stream, xx, \
                       ldx, w.cols, w.had, w.sv, offsets, w.groups, r0, xh, xs)
    const int64_t per = rows_a_launch(512);
    for (int64_t r0 = 0; r0 < n; r0 += per) {
        const unsigned rows = (unsigned)(n - r0 < per ? n - r0 : per);
        // a round a row while that takes at most 512 lanes
        if (bf16 && w.cols <= 2048)
            EXL3_ROTATE(true, 256);
        else if (bf16)
            EXL3_ROTATE(true, 512);
        else if (w.cols <= 2048)
            EXL3_ROTATE(false, 256);
        else
            EXL3_ROTATE(false, 512);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
#undef EXL3_ROTATE
    return hipSuccess;
}

hipError_t launch_coded_rows(const WeightArgs &w, const int32_t *offsets, const RowsArgs &a,
                             hipStream_t stream) {
#define EXL3_ROWS_K(LV, KK) \
    case KK: return coded_rows_t<LV, KK>(w, offsets, a, stream)
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
    return coded_rows_t<kLevelsTable, 0>(w, offsets, a, stream);
}

hipError_t launch_coded_tiles(const WeightArgs &w, const int32_t *offsets, const uint16_t *xh,
                              const float *xs, int64_t n, bool transposed, int per, int split,
                              float *part, bool bf16, const AdapterArgs *ad, const uint16_t *v, void *y,
                              int64_t ldy, hipStream_t stream) {
    // one split: the kernel finishes y
    const TilesOut out{w.scale, w.su, w.had, ad ? *ad : AdapterArgs{}, v, bf16,
                       split == 1 ? static_cast<uint16_t *>(y) : nullptr, ldy};
    const int row_blocks = (w.rows + 127) / 128;
    const int64_t n_tiles = offsets ? n / per + w.groups : (n + per - 1) / per;
    const int total = (int)(n_tiles * row_blocks * split);
#define EXL3_TILES_T(LV, KK, NT, T)                                                             \
    hipLaunchKernelGGL((coded_tiles_kernel<LV, KK, NT, T>), dim3((unsigned)total), dim3(256),   \
                       0, stream, w.packed, w.lv, w.rows, w.cols, offsets, w.groups, xh, xs, n, \
                       split, row_blocks, total, part, out)
#define EXL3_TILES_NT(LV, KK, NT)                                                               \
    do {                                                                                        \
        if (transposed)                                                                         \
            EXL3_TILES_T(LV, KK, NT, true);                                                     \
        else                                                                                    \
            EXL3_TILES_T(LV, KK, NT, false);                                                    \
    } while (0)
#define EXL3_TILES(LV, KK)                                                                      \
    case KK:                                                                                    \
        if (per == 32)                                                                          \
            EXL3_TILES_NT(LV, KK, 2);                                                           \
        else if (per == 64)                                                                     \
            EXL3_TILES_NT(LV, KK, 4);                                                           \
        else                                                                                    \
            EXL3_TILES_NT(LV, KK, 8);                                                           \
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
#undef EXL3_TILES_NT
#undef EXL3_TILES_T
    return hipGetLastError();
}

hipError_t launch_finish(const WeightArgs &w, const int32_t *offsets, const float *part, int split,
                         int64_t n, bool bf16, const AdapterArgs *ad, const uint16_t *v, void *y,
                         int64_t ldy, hipStream_t stream) {
    const int blocks = (w.rows + 511) / 512;
    const AdapterArgs args = ad ? *ad : AdapterArgs{};
    const int64_t per = rows_a_launch(64 * blocks);
    for (int64_t t0 = 0; t0 < n; t0 += per) {
        const unsigned grid = (unsigned)(n - t0 < per ? n - t0 : per) * (unsigned)blocks;
        hipLaunchKernelGGL(finish_kernel, dim3(grid), dim3(64), 0, stream, part, split, n, w.rows,
                           w.had, w.scale, w.su, offsets, w.groups, args, v, bf16, t0,
                           static_cast<uint16_t *>(y), ldy);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace exl3
