// Low-rank adapters beside a coded projection on gfx950: the products with the
// narrow matrices.  A row t of the activations has the adapter a = ids[t] (or
// none), and v_t = alpha_a A_a x_t enters the projection's kernels as one
// more, short, contraction (B_a v_t).  v is rounded to the activations' type,
// as the operand of that product: at most 2^-8 (bfloat16) or 2^-11 (binary16) of
// each value, the adapter's part of a result that is rounded to the same type.
// Binary16's range would cut gradients of common sizes (dy of 1e-5 and B of 1e-3
// give u = alpha B^T dy near its least step), so there each row is stored over a
// power of two that takes its largest value into [2^13, 2^14).
#include "coded.h"

namespace exl3 {

namespace {

// Eight consecutive 16-bit elements, on any two bytes.
__device__ __forceinline__ u32x4 load8(const uint16_t *p) {
    return *reinterpret_cast<const u32x4u *>(p);
}

// ---- v = alpha A x ----
// A workgroup per 16 rows of x, and in grid.y the share of the rows' distinct
// adapters it takes in turn (many requests: one each, so that they run beside
// each other; long prompts: one or two shares).  The waves take 32 U columns of
// the contraction at a time and their sums meet in shared memory.  The matrix
// instruction multiplies all 16 rows by each adapter and keeps those that have
// it: its rate is far from the bound, which is what one compute unit can have
// under way of its misses, about 15 bytes a cycle: x and A for 16 rows, 4,096
// columns, take 10 us at rank 16 and 21 us at rank 64, and neither loads in
// larger groups (21 us) nor a workgroup for each 16 ranks (24 us) nor the
// contraction in two workgroups (16 us with one adapter, 25 us with eight) nor
// rows of one adapter on one die (as without) shorten them.  grid.z: up to two
// such products.
template <bool BF, int RT>
__global__ void __launch_bounds__(512)
shrink_kernel(AdapterArgs ad, ShrinkArgs p0, ShrinkArgs p1, int64_t n) {
    constexpr int kWaves = 8;
    __shared__ f32x4 sums[kWaves][RT][64];
    __shared__ uint32_t row_big[RT][16];
    const ShrinkArgs p = blockIdx.z ? p1 : p0;
    const int lane = threadIdx.x & 63, wv = wave_number();
    const int r = lane & 15, g = lane >> 4, k = p.k;
    const int64_t t0 = (int64_t)blockIdx.x * 16;
    const int64_t tok = t0 + r < n ? t0 + r : n - 1;
    int id_r = t0 + r < n ? ad.ids[tok] : -1;    // of the lane's row; -1: none
    if (id_r < 0 || id_r >= ad.count) id_r = -1;
    // rows that are the first of their adapter
    bool seen = id_r < 0 || lane >= 16;
#pragma unroll
    for (int q = 0; q < 15; ++q) {
        const int other = __shfl(id_r, q);
        seen |= q < r && other == id_r;
    }
    uint32_t firsts = (uint32_t)__ballot(!seen) & 0xFFFFu;
    if (blockIdx.y == 0) {
        // rows without an adapter, and the padding that no tile of ranks covers
        for (int c = 16 * RT + 4 * (wv * 4 + g); c < ad.rank_pad; c += 16 * kWaves)
            if (t0 + r < n) *reinterpret_cast<uint2 *>(p.v + tok * ad.rank_pad + c) = uint2{0u, 0u};
        for (int c = 4 * (wv * 4 + g); c < ad.rank_pad; c += 16 * kWaves)
            if (t0 + r < n && id_r < 0)
                *reinterpret_cast<uint2 *>(p.v + tok * ad.rank_pad + c) = uint2{0u, 0u};
    }
    const uint16_t *xr = p.x + tok * p.ldx + 8 * g;
    uint32_t turn = 0;
    for (; firsts; firsts &= firsts - 1, ++turn) {
        if ((turn & (gridDim.y - 1)) != blockIdx.y) continue;      // gridDim.y: a power of two
        const int id = __shfl(id_r, __ffs(firsts) - 1);
        const uint16_t *ar = p.a + (size_t)id * ad.rank * k + 8 * g;
        uint32_t row_at[RT];                     // past the rank: the last, made zero
#pragma unroll
        for (int t = 0; t < RT; ++t)
            row_at[t] = (uint32_t)(16 * t + r < ad.rank ? 16 * t + r : ad.rank - 1) * (uint32_t)k;
        f32x4 acc[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        constexpr int U = RT <= 2 ? 4 : 2;
        const u32x4 zero = {0u, 0u, 0u, 0u};
        for (int c0 = wv * 32 * U; c0 < k; c0 += 32 * kWaves * U) {
            // all loads at once; past the end they repeat the first step's, made zero
            u32x4 xv[U], av[U][RT];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int c = c0 + 32 * j < k ? c0 + 32 * j : c0;
                xv[j] = load8(xr + c);
#pragma unroll
                for (int t = 0; t < RT; ++t) av[j][t] = load8(ar + row_at[t] + c);
            }
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const bool in = c0 + 32 * j < k;
                const u32x4 xj = in ? xv[j] : zero;
#pragma unroll
                for (int t = 0; t < RT; ++t)
                    acc[t] = Act<BF>::mfma(in && 16 * t + r < ad.rank ? av[j][t] : zero, xj, acc[t]);
            }
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) sums[wv][t][lane] = acc[t];
        __syncthreads();
        f32x4 z;
        if (wv < RT) {                           // a wave a tile of ranks
            z = sums[0][wv][lane];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) z += sums[w][wv][lane];
            z = ad.alpha[id] * z;
            if (!BF) {
                // the row's largest finite magnitude (as an integer; the others go
                // their own way)
                uint32_t big = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float zi = z[i];       // (a bit cast of z[i] itself is z[0]'s)
                    const uint32_t m = __builtin_bit_cast(uint32_t, zi) & 0x7FFFFFFFu;
                    big = id_r == id && m < 0x7F800000u && m > big ? m : big;
                }
#pragma unroll
                for (int s = 16; s < 64; s <<= 1) {
                    const uint32_t o = (uint32_t)__shfl_xor((int)big, s);
                    big = o > big ? o : big;
                }
                if (lane < 16) row_big[wv][lane] = big;
            }
        }
        if (!BF) __syncthreads();
        if (wv < RT) {
            PowerOfTwo one{1.0f, 1.0f, 1.0f, false}, all = one;      // of the row, and of 16
            if (!BF) {
                uint32_t big = row_big[0][r];
#pragma unroll
                for (int t = 1; t < RT; ++t) big = row_big[t][r] > big ? row_big[t][r] : big;
                one = scale_for(big);
#pragma unroll
                for (int s = 1; s < 16; s <<= 1) {
                    const uint32_t o = (uint32_t)__shfl_xor((int)big, s);
                    big = o > big ? o : big;
                }
                all = scale_for(big);
            }
            auto pair = [&](const PowerOfTwo &p2, int i) {
                return BF ? Act<BF>::store2(z[i], z[i + 1])
                          : Act<BF>::store2(z[i] * p2.up * p2.up2, z[i + 1] * p2.up * p2.up2);
            };
            const int c = 16 * wv + 4 * g;
            if (id_r == id && c < ad.rank_pad) {
                *reinterpret_cast<uint2 *>(p.v + tok * ad.rank_pad + c) =
                    uint2{pair(one, 0), pair(one, 2)};
                if (!BF && c == 0) {
                    if (p.vs) p.vs[tok] = one.scale;
                    if (p.ts) p.ts[tok] = all.scale;
                }
                if (p.vt) {
                    const uint32_t lo = pair(all, 0), hi = pair(all, 2);
                    uint16_t *o = p.vt + (size_t)c * p.ldvt + tok;
                    o[0] = (uint16_t)lo;
                    o[p.ldvt] = (uint16_t)(lo >> 16);
                    o[2 * p.ldvt] = (uint16_t)hi;
                    o[3 * p.ldvt] = (uint16_t)(hi >> 16);
                }
            }
        }
        __syncthreads();
    }
}

// [count][p][q] -> [count][q][p] for up to two arrays (grid.y: count; grid.z: arrays).
// Latency bounds it: 4.7 us for four matrices of 16 x 4096 on each side.
__global__ void __launch_bounds__(256)
transpose16_kernel(TransposeArgs t0, TransposeArgs t1) {
    __shared__ uint16_t tile[32][33];
    const TransposeArgs t = blockIdx.z ? t1 : t0;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int across = (t.q + 31) / 32, down = (t.p + 31) / 32;
    if ((int)blockIdx.x >= across * down) return;
    const size_t at = (size_t)blockIdx.y * t.p * t.q;
    const int q0 = blockIdx.x % across * 32, p0 = blockIdx.x / across * 32;
    for (int i = ty; i < 32; i += 8)
        if (p0 + i < t.p && q0 + tx < t.q)
            tile[i][tx] = t.src[at + (size_t)(p0 + i) * t.q + q0 + tx];
    __syncthreads();
    for (int i = ty; i < 32; i += 8)
        if (q0 + i < t.q && p0 + tx < t.p)
            t.dst[at + (size_t)(q0 + i) * t.p + p0 + tx] = tile[tx][i];
}

// ---- gradients of the adapters' matrices ----
// sum over the rows t of adapter a of u[t][i] q[t][j]: the contraction runs over
// rows, 32 a step.  u comes transposed, so its operand is one load; of q a lane
// loads four neighbouring columns of its eight rows and pairs the rows up in
// registers, which gives the operands of four tiles of 16 columns (columns
// 4 r + c of tile c).  Rows of other adapters enter as zeros on both sides,
// chosen and not multiplied, so that whatever they hold stays out; blocks of
// 32 rows without the adapter are passed over.  The rows are split in parts,
// those that have the adapter are summed in order afterwards: the result does
// not depend on scheduling.  In binary16 the two halves of a block have each a
// power of two of their own for u: the lesser half is brought to the other's, and
// the block's products are added under that.  2,048 rows, four adapters of rank 16, 4096 x 4096:
// 17.5 us for both matrices, x and dy read once, eight bytes a lane and load, which
// bounds it (34 MB, 1.9 TB/s).
// grid: blocks of 256 columns of the first product, then of the second;
// adapters; parts.
constexpr int kGradBlocks = 16;            // blocks of 32 rows whose adapters are read at once

template <bool BF, int RT>
__global__ void __launch_bounds__(256)
adapter_grad_kernel(AdapterArgs ad, GradArgs g0, GradArgs g1, int64_t n, int64_t per_split,
                    uint8_t *__restrict__ used) {
    const int lane = threadIdx.x & 63, wv = wave_number();
    const int r = lane & 15, g = lane >> 4, id = blockIdx.y;
    const int first = (g0.k + 255) / 256;
    const bool second = (int)blockIdx.x >= first;
    const GradArgs p = second ? g1 : g0;
    const int j0 = ((int)blockIdx.x - (second ? first : 0)) * 256 + wv * 64;
    if (j0 >= p.k) return;
    const int64_t t_lo = blockIdx.z * per_split;
    const int64_t t_hi = t_lo + per_split < n ? t_lo + per_split : n;
    f32x4 acc[RT][4];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[t][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const uint16_t *qc = p.q + j0 + 4 * r;

    struct Step {
        uint2 x[8];
        u32x4 u[RT];
        uint32_t has;
        float half[2];                           // the halves' powers of two (binary16)
    };
    auto fetch = [&](Step &s, int64_t b, uint32_t has) {
        s.has = has;
        if (!BF) {
            const uint32_t lo = has & 0xFFFFu, hi = has >> 16;
            s.half[0] = lo ? p.us[b + __ffs(lo) - 1] : 0.0f;
            s.half[1] = hi ? p.us[b + 16 + __ffs(hi) - 1] : 0.0f;
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            s.x[t] = uint2{0u, 0u};
            if ((has >> (8 * g + t)) & 1u) {
                const uint16_t *at = qc + (b + 8 * g + t) * p.ldq;
                const u32x2u two = *reinterpret_cast<const u32x2u *>(at);
                s.x[t] = uint2{two[0], two[1]};
            }
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            s.u[t] = u32x4{0u, 0u, 0u, 0u};
            if (16 * t + r < ad.rank)
                s.u[t] = *reinterpret_cast<const u32x4 *>(p.ut + (size_t)(16 * t + r) * p.ldut + b +
                                                          8 * g);
        }
    };
    auto use = [&](Step &s) {
        u32x4 keep;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t two = (s.has >> (8 * g + 2 * c)) & 3u;
            keep[c] = (two & 1u ? 0xFFFFu : 0u) | (two & 2u ? 0xFFFF0000u : 0u);
        }
        u32x4 b[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t ax = s.x[2 * c].x, bx = s.x[2 * c + 1].x;
            const uint32_t ay = s.x[2 * c].y, by = s.x[2 * c + 1].y;
            b[0][c] = __builtin_amdgcn_perm(bx, ax, 0x05040100u);
            b[1][c] = __builtin_amdgcn_perm(bx, ax, 0x07060302u);
            b[2][c] = __builtin_amdgcn_perm(by, ay, 0x05040100u);
            b[3][c] = __builtin_amdgcn_perm(by, ay, 0x07060302u);
        }
        if (BF) {
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const u32x4 u = s.u[t] & keep;
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[t][c] = Act<BF>::mfma(u, b[c], acc[t][c]);
            }
        } else {
            const float up = s.half[0] > s.half[1] ? s.half[0] : s.half[1];
            const _Float16 by = (_Float16)((g < 2 ? s.half[0] : s.half[1]) / up);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const u32x4 u = __builtin_bit_cast(
                    u32x4, __builtin_bit_cast(f16x8, s.u[t] & keep) * by);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const f32x4 z = Act<BF>::mfma(u, b[c], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[t][c][i] = __builtin_fmaf(z[i], up, acc[t][c][i]);
                }
            }
        }
    };
    bool any = false;
    for (int64_t c0 = t_lo; c0 < t_hi; c0 += 32 * kGradBlocks) {
        // which rows of each block have the adapter: bits of 16 words, one a lane
        uint32_t mine = 0;
#pragma unroll
        for (int b = 0; b < kGradBlocks; b += 2) {
            const int64_t t = c0 + 32 * b + lane;
            const uint64_t has = __ballot(t < t_hi && ad.ids[t] == id);
            if (lane == b) mine = (uint32_t)has;
            if (lane == b + 1) mine = (uint32_t)(has >> 32);
        }
        uint64_t left = __ballot(mine != 0);
        if (!left) continue;
        any = true;
        Step s[2];
        int b = __ffsll((unsigned long long)left) - 1;
        left &= left - 1;
        fetch(s[0], c0 + 32 * b, __builtin_amdgcn_readlane(mine, b));
        while (left) {
            b = __ffsll((unsigned long long)left) - 1;
            left &= left - 1;
            fetch(s[1], c0 + 32 * b, __builtin_amdgcn_readlane(mine, b));
            use(s[0]);
            s[0] = s[1];
        }
        use(s[0]);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) used[blockIdx.z * ad.count + id] = any;
    if (!any) return;
    // column j0 + 4 r + c, ranks 16 t + 4 g ..
    float *o = p.part + ((size_t)blockIdx.z * ad.count + id) * ad.rank * p.k;
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int rank = 16 * t + 4 * g + i;
            if (rank >= ad.rank) continue;
            if (p.transposed) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    o[(size_t)(j0 + 4 * r + c) * ad.rank + rank] = acc[t][c][i];
            } else {
                *reinterpret_cast<f32x4 *>(o + (size_t)rank * p.k + j0 + 4 * r) =
                    f32x4{acc[t][0][i], acc[t][1][i], acc[t][2][i], acc[t][3][i]};
            }
        }
}

// The parts' sums of both products (grid.y), four elements a thread.  5 us for 16
// parts of the above.
template <bool BF>
__global__ void __launch_bounds__(256)
adapter_sum_kernel(GradArgs g0, GradArgs g1, int splits, int count, int rank, size_t first,
                   const uint8_t *__restrict__ used) {
    const GradArgs p = blockIdx.y ? g1 : g0;
    const size_t all = (size_t)count * rank * p.k;
    const size_t i = first + ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= all) return;
    const int id = (int)(i / ((size_t)rank * p.k));
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
    // eight parts' loads under way at a time
    for (int q0 = 0; q0 < splits; q0 += 8) {
        bool has[8];
        f32x4 v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) has[q] = q0 + q < splits && used[(q0 + q) * count + id];
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (has[q]) v[q] = *reinterpret_cast<const f32x4 *>(p.part + (q0 + q) * all + i);
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (has[q]) s += v[q];
    }
    *reinterpret_cast<u32x2u *>(p.out + i) =
        u32x2u{Act<BF>::store2(s[0], s[1]), Act<BF>::store2(s[2], s[3])};
}

}  // namespace

hipError_t launch_shrink(const AdapterArgs &ad, const ShrinkArgs *p, int products, int64_t n,
                         bool bf16, hipStream_t stream) {
    ShrinkArgs q[2];
    for (int i = 0; i < 2; ++i) q[i] = p[i < products ? i : 0];
    const unsigned tiles = (unsigned)((n + 15) / 16);
    // up to 16 distinct adapters a tile: a workgroup each while all workgroups run
    // at once (two a compute unit; those without work would hold up the others)
    unsigned share = 16;
    while (share > 1 && tiles * share * (unsigned)products > 512) share /= 2;
    const dim3 grid(tiles, share, (unsigned)products);
#define EXL3_SHRINK(RT)                                                                     \
    do {                                                                                    \
        if (bf16)                                                                           \
            hipLaunchKernelGGL((shrink_kernel<true, RT>), grid, dim3(512), 0, stream, ad, q[0], \
                               q[1], n);                                                    \
        else                                                                                \
            hipLaunchKernelGGL((shrink_kernel<false, RT>), grid, dim3(512), 0, stream, ad, q[0],\
                               q[1], n);                                                    \
    } while (0)
    if (ad.rank <= 16)
        EXL3_SHRINK(1);
    else if (ad.rank <= 32)
        EXL3_SHRINK(2);
    else if (ad.rank <= 64)
        EXL3_SHRINK(4);
    else
        EXL3_SHRINK(8);
#undef EXL3_SHRINK
    return hipGetLastError();
}

hipError_t launch_transpose16(const TransposeArgs *t, int arrays, int count, hipStream_t stream) {
    const TransposeArgs &a = t[0], &b = t[arrays - 1];
    const unsigned ta = (unsigned)((a.p + 31) / 32) * (unsigned)((a.q + 31) / 32);
    const unsigned tb = (unsigned)((b.p + 31) / 32) * (unsigned)((b.q + 31) / 32);
    hipLaunchKernelGGL(transpose16_kernel,
                       dim3(ta > tb ? ta : tb, (unsigned)count, (unsigned)arrays), dim3(256), 0,
                       stream, a, b);
    return hipGetLastError();
}

int adapter_grad_splits(int64_t n, int count) {
    // parts of 128 rows, up to 32 of them; many adapters fill the chip with fewer
    const int64_t s = (n + 127) / 128, most = 128 / count;
    return (int)(s < 1 || most < 1 ? 1 : s < most ? (s < 32 ? s : 32) : most < 32 ? most : 32);
}

hipError_t launch_adapter_grad(const AdapterArgs &ad, const GradArgs *p, int products, int64_t n,
                               bool bf16, int splits, uint8_t *used, hipStream_t stream) {
    GradArgs q[2];
    for (int i = 0; i < 2; ++i) q[i] = p[i < products ? i : 0];
    const int64_t per = ((n + splits - 1) / splits + 31) / 32 * 32;
    const int blocks = (q[0].k + 255) / 256 + (products > 1 ? (q[1].k + 255) / 256 : 0);
    const dim3 grid((unsigned)blocks, (unsigned)ad.count, (unsigned)splits);
#define EXL3_GRAD(RT)                                                                       \
    do {                                                                                    \
        if (bf16)                                                                           \
            hipLaunchKernelGGL((adapter_grad_kernel<true, RT>), grid, dim3(256), 0, stream, \
                               ad, q[0], q[1], n, per, used);                               \
        else                                                                                \
            hipLaunchKernelGGL((adapter_grad_kernel<false, RT>), grid, dim3(256), 0, stream,\
                               ad, q[0], q[1], n, per, used);                               \
    } while (0)
    if (ad.rank <= 16)
        EXL3_GRAD(1);
    else if (ad.rank <= 32)
        EXL3_GRAD(2);
    else if (ad.rank <= 64)
        EXL3_GRAD(4);
    else
        EXL3_GRAD(8);
#undef EXL3_GRAD
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const int k = q[0].k > q[1].k ? q[0].k : q[1].k;
    const int64_t all = ((int64_t)ad.count * ad.rank * k / 4 + 255) / 256, each = rows_a_launch(256);
    for (int64_t g = 0; g < all; g += each) {
        const dim3 blocks_here((unsigned)(all - g < each ? all - g : each), (unsigned)products);
        const size_t first = (size_t)g * 1024;
        if (bf16)
            hipLaunchKernelGGL((adapter_sum_kernel<true>), blocks_here, dim3(256), 0, stream, q[0],
                               q[1], splits, ad.count, ad.rank, first, used);
        else
            hipLaunchKernelGGL((adapter_sum_kernel<false>), blocks_here, dim3(256), 0, stream,
                               q[0], q[1], splits, ad.count, ad.rank, first, used);
        err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace exl3
