// Low-rank adapters beside a coded projection on gfx950: the products with the
// narrow matrices.  A row t of the activations has the adapter a = ids[t] (or
// none), and v_t = alpha_a A_a x_t enters the projection's kernels as one
// more, short, contraction (B_a v_t).  v is rounded to the activations' type,
// as the operand of that product: 2^-9 (bfloat16) or 2^-12 (binary16) of the
// adapter's part of the result, which is rounded to the same type.
#include "coded.h"

namespace exl3 {

namespace {

// Eight consecutive 16-bit elements; `wide` where they start on 16 bytes.
__device__ __forceinline__ u32x4 load8(const uint16_t *p, bool wide) {
    if (wide) return *reinterpret_cast<const u32x4 *>(p);
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
    return o;
}

// ---- v = alpha A x ----
// A workgroup per 16 rows of x, and in grid.y the share of the rows' distinct
// adapters it takes in turn (many requests: one each, so that they run beside
// each other; long prompts: one share).  Eight waves split the contraction
// and their sums meet in shared memory.  The matrix instruction multiplies
// all 16 rows by each adapter and keeps those that have it: its rate is far
// from the bound, which is reading A once per 16 rows.
template <bool BF, int RT>
__global__ void __launch_bounds__(512)
shrink_kernel(AdapterArgs ad, const uint16_t *__restrict__ a, const uint16_t *__restrict__ x,
              int64_t ldx, int64_t n, int k, bool wide_a, bool wide_x,
              uint16_t *__restrict__ v) {
    __shared__ f32x4 sums[8][RT][64];
    __shared__ int ids[16];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int r = lane & 15, g = lane >> 4;
    const int64_t t0 = (int64_t)blockIdx.x * 16;
    if (threadIdx.x < 16) {
        const int64_t tok = t0 + threadIdx.x;
        const int id = tok < n ? ad.ids[tok] : -1;
        ids[threadIdx.x] = id >= 0 && id < ad.count ? id : -1;
    }
    __syncthreads();
    if (blockIdx.y == 0) {
        for (int i = threadIdx.x; i < 16 * ad.rank_pad; i += 512) {
            const int t = i / ad.rank_pad;
            if (t0 + t < n && ids[t] < 0) v[(t0 + t) * ad.rank_pad + i % ad.rank_pad] = 0;
        }
    }
    const int64_t tok = t0 + r < n ? t0 + r : n - 1;
    const uint16_t *xr = x + tok * ldx + 8 * g;
    int turn = 0;
    for (int s = 0; s < 16; ++s) {
        const int id = ids[s];
        bool seen = id < 0;
        for (int q = 0; q < s; ++q) seen |= ids[q] == id;
        if (seen) continue;
        if (turn++ % (int)gridDim.y != (int)blockIdx.y) continue;
        const uint16_t *ar = a + (size_t)id * ad.rank * k + 8 * g;
        f32x4 acc[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int c = wv * 32; c < k; c += 256) {
            const u32x4 xv = load8(xr + c, wide_x);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                u32x4 av = {0u, 0u, 0u, 0u};
                if (16 * t + r < ad.rank) av = load8(ar + (size_t)(16 * t + r) * k + c, wide_a);
                acc[t] = Act<BF>::mfma(av, xv, acc[t]);
            }
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) sums[wv][t][lane] = acc[t];
        __syncthreads();
        for (int i = threadIdx.x; i < RT * 64; i += 512) {
            const int t = i >> 6, l = i & 63;
            f32x4 z = sums[0][t][l];
#pragma unroll
            for (int w = 1; w < 8; ++w) z += sums[w][t][l];
            const int c = 16 * t + 4 * (l >> 4);
            if (ids[l & 15] == id && c < ad.rank_pad) {
                const float al = ad.alpha[id];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[(t0 + (l & 15)) * ad.rank_pad + c + j] = Act<BF>::store(al * z[j]);
            }
        }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(256)
transpose16_kernel(const uint16_t *__restrict__ src, int p, int q, uint16_t *__restrict__ dst) {
    __shared__ uint16_t tile[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const size_t at = (size_t)blockIdx.z * p * q;
    const int q0 = blockIdx.x * 32, p0 = blockIdx.y * 32;
    for (int i = ty; i < 32; i += 8)
        if (p0 + i < p && q0 + tx < q) tile[i][tx] = src[at + (size_t)(p0 + i) * q + q0 + tx];
    __syncthreads();
    for (int i = ty; i < 32; i += 8)
        if (q0 + i < q && p0 + tx < p) dst[at + (size_t)(q0 + i) * p + p0 + tx] = tile[tx][i];
}

// ---- gradients of the adapters' matrices ----
// sum over the rows t of adapter a of u[t][i] q[t][j], 32 rows a step.  Rows of
// other adapters enter as zeros on both sides, chosen and not multiplied, so
// that whatever they hold stays out.  The rows are split in `splits` parts,
// summed in order afterwards: the result does not depend on scheduling.
template <bool BF, int RT>
__global__ void __launch_bounds__(256)
adapter_grad_kernel(AdapterArgs ad, const uint16_t *__restrict__ u,
                    const uint16_t *__restrict__ q, int64_t ldq, int64_t n, int k,
                    int64_t per_split, float *__restrict__ part) {
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int r = lane & 15, g = lane >> 4;
    const int id = blockIdx.y, j = blockIdx.x * 64 + wv * 16 + r;
    const int64_t t_lo = blockIdx.z * per_split;
    const int64_t t_hi = t_lo + per_split < n ? t_lo + per_split : n;
    f32x4 acc[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t t0 = t_lo; t0 < t_hi; t0 += 32) {
        const int64_t mine = t0 + (lane & 31);
        const uint32_t has = (uint32_t)__ballot(mine < t_hi && ad.ids[mine] == id);
        if (!has) continue;
        u32x4 b;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t w = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int t = 8 * g + 2 * c + h;
                if ((has >> t) & 1u) w |= (uint32_t)q[(t0 + t) * ldq + j] << (16 * h);
            }
            b[c] = w;
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            u32x4 a;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t w = 0;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int t = 8 * g + 2 * c + h;
                    if (((has >> t) & 1u) && 16 * rt + r < ad.rank)
                        w |= (uint32_t)u[(t0 + t) * ad.rank_pad + 16 * rt + r] << (16 * h);
                }
                a[c] = w;
            }
            acc[rt] = Act<BF>::mfma(a, b, acc[rt]);
        }
    }
    float *o = part + ((size_t)blockIdx.z * ad.count + id) * ad.rank * k;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int i = 16 * rt + 4 * g + c;
            if (i < ad.rank) o[(size_t)i * k + j] = acc[rt][c];
        }
}

template <bool BF>
__global__ void __launch_bounds__(256)
adapter_sum_kernel(const float *__restrict__ part, int splits, int count, int rank, int k,
                   bool transposed, uint16_t *__restrict__ out) {
    const size_t all = (size_t)count * rank * k, i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= all) return;
    size_t from = i;
    if (transposed) {                    // out is [count][k][rank]
        const size_t a = i / ((size_t)rank * k), rest = i - a * rank * k;
        from = (a * rank + rest % rank) * k + rest / rank;
    }
    float s = 0.0f;
    for (int p = 0; p < splits; ++p) s += part[(size_t)p * all + from];
    out[i] = Act<BF>::store(s);
}

}  // namespace

hipError_t launch_shrink(const AdapterArgs &ad, const void *a, const void *x, int64_t ldx,
                         int64_t n, int k, bool bf16, uint16_t *v, hipStream_t stream) {
    const unsigned tiles = (unsigned)((n + 15) / 16);
    // up to 16 distinct adapters a tile: a workgroup each while there are few tiles
    const dim3 grid(tiles, tiles <= 32 ? 16u : tiles <= 128 ? 4u : 1u);
    const bool wide_a = reinterpret_cast<uintptr_t>(a) % 16 == 0;
    const bool wide_x = reinterpret_cast<uintptr_t>(x) % 16 == 0 && ldx % 8 == 0;
    const uint16_t *aa = static_cast<const uint16_t *>(a), *xx = static_cast<const uint16_t *>(x);
#define EXL3_SHRINK(RT)                                                                      \
    do {                                                                                     \
        if (bf16)                                                                            \
            hipLaunchKernelGGL((shrink_kernel<true, RT>), grid, dim3(512), 0, stream, ad, aa, \
                               xx, ldx, n, k, wide_a, wide_x, v);                            \
        else                                                                                 \
            hipLaunchKernelGGL((shrink_kernel<false, RT>), grid, dim3(512), 0, stream, ad, aa, \
                               xx, ldx, n, k, wide_a, wide_x, v);                            \
    } while (0)
    if (ad.rank_pad <= 32)
        EXL3_SHRINK(2);
    else if (ad.rank_pad <= 64)
        EXL3_SHRINK(4);
    else
        EXL3_SHRINK(8);
#undef EXL3_SHRINK
    return hipGetLastError();
}

hipError_t launch_transpose16(const void *src, int count, int p, int q, void *dst,
                              hipStream_t stream) {
    const dim3 grid((unsigned)((q + 31) / 32), (unsigned)((p + 31) / 32), (unsigned)count);
    hipLaunchKernelGGL(transpose16_kernel, grid, dim3(256), 0, stream,
                       static_cast<const uint16_t *>(src), p, q, static_cast<uint16_t *>(dst));
    return hipGetLastError();
}

int adapter_grad_splits(int64_t n, int k, int count) {
    // about two workgroups a compute unit, of 128 rows at least
    const int64_t groups = (int64_t)(k / 64) * count;
    int64_t s = 512 / groups;
    if (s > (n + 127) / 128) s = (n + 127) / 128;
    return s < 1 ? 1 : (int)s;
}

hipError_t launch_adapter_grad(const AdapterArgs &ad, const uint16_t *u, const void *q,
                               int64_t ldq, int64_t n, int k, bool bf16, bool transposed,
                               int splits, float *part, void *out, hipStream_t stream) {
    const int64_t per = ((n + splits - 1) / splits + 31) / 32 * 32;
    const dim3 grid((unsigned)(k / 64), (unsigned)ad.count, (unsigned)splits);
    const uint16_t *qq = static_cast<const uint16_t *>(q);
#define EXL3_GRAD(RT)                                                                          \
    do {                                                                                       \
        if (bf16)                                                                              \
            hipLaunchKernelGGL((adapter_grad_kernel<true, RT>), grid, dim3(256), 0, stream, ad, \
                               u, qq, ldq, n, k, per, part);                                   \
        else                                                                                   \
            hipLaunchKernelGGL((adapter_grad_kernel<false, RT>), grid, dim3(256), 0, stream,   \
                               ad, u, qq, ldq, n, k, per, part);                               \
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
    const size_t all = (size_t)ad.count * ad.rank * k;
    const unsigned blocks = (unsigned)((all + 255) / 256);
    uint16_t *o = static_cast<uint16_t *>(out);
    if (bf16)
        hipLaunchKernelGGL((adapter_sum_kernel<true>), dim3(blocks), dim3(256), 0, stream, part,
                           splits, ad.count, ad.rank, k, transposed, o);
    else
        hipLaunchKernelGGL((adapter_sum_kernel<false>), dim3(blocks), dim3(256), 0, stream, part,
                           splits, ad.count, ad.rank, k, transposed, o);
    return hipGetLastError();
}

}  // namespace exl3
