// Root-mean-square norm with the residual's addition, its backward pass, and the writing of
// activations and matrices as 8-bit blocks (gfx950).  All of them are bound by memory: each
// element is read once, kept in registers between the reductions, and written once.
#include "blocks.h"

#include "exl3.h"

namespace exl3 {

namespace {

// Eight factors of the gain at column c.
template <bool BF, bool G32>
__device__ __forceinline__ void load_gain(const void *gain, int c, int valid, float (&f)[kWide]) {
    if (G32) {
        const float *p = static_cast<const float *>(gain) + c;
        if (valid >= kWide) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const f32x4 v = *reinterpret_cast<const f32x4u *>(p + 4 * h);
#pragma unroll
                for (int i = 0; i < 4; ++i) f[4 * h + i] = v[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < kWide; ++i) f[i] = i < valid ? p[i] : 0.0f;
        }
    } else {
        widen<BF>(load8(static_cast<const uint16_t *>(gain) + c, valid), f);
    }
}

// Sum over the workgroup's lanes, the same in all of them and in a fixed order.
template <int T, typename S>
__device__ __forceinline__ S sum_all(S v, S *between) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
    if (T == 64) return v;
    __syncthreads();                             // the last use of `between` is over
    if ((threadIdx.x & 63) == 0) between[threadIdx.x >> 6] = v;
    __syncthreads();
    v = between[0];
#pragma unroll
    for (int w = 1; w < T / 64; ++w) v += between[w];
    return v;
}

// Eight columns from c of a row of blocks: the block's scale by its first lane, the codes by all,
// zeros past the width up to whole blocks.  All 16 lanes of a block take part.
__device__ __forceinline__ void write_codes(const BlockRowsArgs &q, int64_t row, int c, int cols,
                                            const float (&f)[kWide]) {
    const CodeScale s = code_scale(largest_of_block(largest8(f)));
    if (c >= blocks_of(cols) * kBlock) return;
    *reinterpret_cast<u32x2 *>(q.q + row * q.ld + c) = first_codes(to_codes(f, s), cols - c);
    if ((c & (kBlock - 1)) == 0) q.scale[(c / kBlock) * q.lds + row] = s.scale;
}

// Two sums at once through places used in turn, so that one barrier serves (a lane is past the
// reads of one place when it writes to it again, as the other's barrier lies between).
template <int T>
__device__ __forceinline__ void sum_both(float &v, float &w, float2 (&between)[2][T / 64],
                                         int &turn) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        v += __shfl_xor(v, m);
        w += __shfl_xor(w, m);
    }
    if (T == 64) return;
    if ((threadIdx.x & 63) == 0) between[turn][threadIdx.x >> 6] = float2{v, w};
    __syncthreads();
    v = between[turn][0].x;
    w = between[turn][0].y;
#pragma unroll
    for (int i = 1; i < T / 64; ++i) {
        v += between[turn][i].x;
        w += between[turn][i].y;
    }
    turn ^= 1;
}

// A sum of squares that binary32 holds: neither too large nor, beside eps, too small.
__device__ __forceinline__ bool in_range(float squares, float eps, int cols) {
    return squares < 0x1p126f && (squares > 0x1p-80f || eps * (float)cols > 0x1p-80f);
}

// 1 / sqrt(mean + eps) as mantissa * 2^exponent: the factor itself, and what it multiplies, may
// lie outside binary32's normal range while their product does not.
struct Rsqrt {
    float mantissa;
    int exponent;
};
__device__ __forceinline__ Rsqrt split(float r) {
    return Rsqrt{__builtin_amdgcn_frexp_mantf(r), __builtin_amdgcn_frexp_expf(r)};
}
__device__ __forceinline__ Rsqrt split(double r) {
    return Rsqrt{(float)__builtin_amdgcn_frexp_mant(r), __builtin_amdgcn_frexp_exp(r)};
}
__device__ __forceinline__ float times(float v, const Rsqrt &r) {
    return __builtin_ldexpf(v, r.exponent) * r.mantissa;
}

// ---- norm ----
// y = s r gain with r = 1 / sqrt(mean(s^2) + eps) and s = x + residual in binary32, before its
// rounding to the stored sum.  A row by T lanes, T / 64 waves; each lane keeps V pieces of eight
// columns.  V = 0: rows too wide for that, which are read twice.  Where the squares leave
// binary32's range the row is summed again in binary64.  Roundings: s to its stored type, y once
// to its type, or its quotient by the block's scale to binary32 and then e4m3.
// 8,200 x 4,096, bfloat16, residual and blocks: 43 us, 5.4 TB/s where a large copy reaches 4.88;
// 1 x 4,096: 2.9 us, the rest of a call's 14.5 is the host's.  1,000 x 20,000 into 16 bits (V = 0):
// 41 (33 the floor).
template <int T, int V, bool BF, bool G32>
__global__ void __launch_bounds__(T < 256 ? 256 : T)
rms_norm_kernel(NormArgs a) {
    constexpr int kRows = T < 256 ? 256 / T : 1; // rows a workgroup
    constexpr int kKeep = V ? V : 1, kUnroll = kKeep;
    __shared__ float between[T / 64];
    __shared__ double between64[T / 64];
    const int lane = T < 256 ? threadIdx.x % T : threadIdx.x;
    const int64_t row = (int64_t)blockIdx.x * kRows + (T < 256 ? threadIdx.x / T : 0);
    if (row >= a.n) return;                      // a whole wave, and no barrier where T = 64
    const uint16_t *x = static_cast<const uint16_t *>(a.x) + row * a.ldx;
    const uint16_t *res = a.residual ? static_cast<const uint16_t *>(a.residual) + row * a.ldr
                                     : nullptr;
    const int pieces = V ? V : (a.cols + T * kWide - 1) / (T * kWide);
    float keep[kKeep][kWide];
    auto load = [&](int i, float (&f)[kWide]) {
        const int c = (i * T + lane) * kWide, valid = a.cols - c;
        widen<BF>(load8(x + c, valid), f);
        if (res) {
            float g[kWide];
            widen<BF>(load8(res + c, valid), g);
#pragma unroll
            for (int j = 0; j < kWide; ++j) f[j] += g[j];
        }
    };
    float squares = 0.0f;
#pragma unroll kUnroll
    for (int i = 0; i < (V ? V : pieces); ++i) {
        load(i, keep[V ? i : 0]);
#pragma unroll
        for (int j = 0; j < kWide; ++j)
            squares = __builtin_fmaf(keep[V ? i : 0][j], keep[V ? i : 0][j], squares);
    }
    squares = sum_all<T>(squares, between);
    Rsqrt r = split(1.0f / sqrtf(squares / (float)a.cols + a.eps));
    if (!in_range(squares, a.eps, a.cols)) {
        double d = 0.0;
#pragma unroll 1
        for (int i = 0; i < pieces; ++i) {
            float f[kWide];
            load(i, f);
#pragma unroll
            for (int j = 0; j < kWide; ++j) d += (double)f[j] * (double)f[j];
        }
        r = split(1.0 / sqrt(sum_all<T>(d, between64) / (double)a.cols + (double)a.eps));
    }
#pragma unroll kUnroll
    for (int i = 0; i < (V ? V : pieces); ++i) {
        const int c = (i * T + lane) * kWide, valid = a.cols - c;
        float f[kWide], g[kWide];
        if (V) {
#pragma unroll
            for (int j = 0; j < kWide; ++j) f[j] = keep[V ? i : 0][j];
        } else {
            load(i, f);
        }
        if (a.sum && valid > 0)
            store8(static_cast<uint16_t *>(a.sum) + row * a.ldsum + c, narrow<BF>(f), valid);
        load_gain<BF, G32>(a.gain, c, valid, g);
#pragma unroll
        for (int j = 0; j < kWide; ++j) f[j] = times(f[j], r) * g[j];
        if (valid < kWide)
#pragma unroll
            for (int j = 0; j < kWide; ++j) f[j] = j < valid ? f[j] : 0.0f;
        if (a.y) {
            if (valid > 0)
                store8(static_cast<uint16_t *>(a.y) + row * a.ldy + c, narrow<BF>(f), valid);
        } else {
            write_codes(a.q, row, c, a.cols, f);
        }
    }
}

// ---- backward ----
// With u = s r and du = dy gain: dx = ds + r (du - u mean(du u)), dgain = sum over rows of dy u.
// A workgroup takes rows blockIdx.x, + parts, ..: one pass over each gives both sums, and the
// gain's gradient of its columns stays in registers until the rows are done.  The parts are
// added in order by a second kernel, so no result depends on scheduling.  V = 0: columns too many
// for registers; dgain goes through the part in memory.  The next row's loads go out before this
// one's sums, whose barrier they would else wait behind: 2,000 x 4,096 with ds: 19.4 us
// a call (13.4 the floor); by the profiler's clock 17.7, then 4.0 for the parts, and 25.8 and 5.0
// with this row's loads behind the last one's sums, 256 lanes a row and one workgroup a compute
// unit.  8,200 rows: 59.3 (55).  1,000 x 20,000 (V = 0): 107 (33).
template <int T, int V, bool BF, bool G32>
__global__ void __launch_bounds__(T)
rms_norm_backward_kernel(NormBackwardArgs a) {
    constexpr int kKeep = V ? V : 1, kUnroll = kKeep;
    __shared__ float2 between[2][T / 64];
    __shared__ double between64[T / 64], between642[T / 64];
    const int lane = threadIdx.x;
    const int pieces = V ? V : (a.cols + T * kWide - 1) / (T * kWide);
    float *part = a.part ? a.part + (int64_t)blockIdx.x * a.cols : nullptr;
    float dg[kKeep][kWide] = {};
    bool first = true;
    int turn = 0;
    u32x4 s8[kKeep], y8[kKeep], d8[kKeep], sn[kKeep], yn[kKeep], dn[kKeep];
    constexpr bool kAhead = V > 0 && T < 1024;   // by a row, where there are registers for it
    auto load_row = [&](int64_t row) {
        const uint16_t *sp = static_cast<const uint16_t *>(a.s) + row * a.lds;
        const uint16_t *yp = static_cast<const uint16_t *>(a.dy) + row * a.lddy;
        const uint16_t *dp = static_cast<const uint16_t *>(a.ds) + row * a.ldds;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * T + lane) * kWide, valid = a.cols - c;
            sn[i] = load8(sp + c, valid);
            yn[i] = load8(yp + c, valid);
            dn[i] = a.ds ? load8(dp + c, valid) : u32x4{0u, 0u, 0u, 0u};
        }
    };
    if (kAhead) load_row(blockIdx.x);
    for (int64_t row = blockIdx.x; row < a.n; row += a.parts) {
        const uint16_t *sp = static_cast<const uint16_t *>(a.s) + row * a.lds;
        const uint16_t *yp = static_cast<const uint16_t *>(a.dy) + row * a.lddy;
        const uint16_t *dp = static_cast<const uint16_t *>(a.ds) + row * a.ldds;
        if (V) {
            if (!kAhead) load_row(row);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                s8[i] = sn[i];
                y8[i] = yn[i];
                d8[i] = dn[i];
            }
            if (kAhead && row + a.parts < a.n) load_row(row + a.parts);
        }
        // (V = 0: read where they are used, twice)
        auto piece = [&](int i, int c, int valid, float (&s)[kWide], float (&y)[kWide],
                         float (&g)[kWide]) {
            load_gain<BF, G32>(a.gain, c, valid, g);
            widen<BF>(V ? s8[V ? i : 0] : load8(sp + c, valid), s);
            widen<BF>(V ? y8[V ? i : 0] : load8(yp + c, valid), y);
        };
        float squares = 0.0f, dot = 0.0f;
#pragma unroll kUnroll
        for (int i = 0; i < (V ? V : pieces); ++i) {
            const int c = (i * T + lane) * kWide, valid = a.cols - c;
            float s[kWide], y[kWide], g[kWide];
            piece(i, c, valid, s, y, g);
#pragma unroll
            for (int j = 0; j < kWide; ++j) {
                squares = __builtin_fmaf(s[j], s[j], squares);
                dot = __builtin_fmaf(y[j] * g[j], s[j], dot);
            }
        }
        sum_both<T>(squares, dot, between, turn);
        const float r32 = 1.0f / sqrtf(squares / (float)a.cols + a.eps);
        Rsqrt r = split(r32);
        float mean = dot * r32 / (float)a.cols;             // of du u
        if (!(in_range(squares, a.eps, a.cols) && magnitude(dot) < 0x7E800000u)) {
            double d = 0.0, e = 0.0;
#pragma unroll 1
            for (int i = 0; i < pieces; ++i) {
                const int c = (i * T + lane) * kWide, valid = a.cols - c;
                float s[kWide], y[kWide], g[kWide];
                load_gain<BF, G32>(a.gain, c, valid, g);
                widen<BF>(load8(sp + c, valid), s);
                widen<BF>(load8(yp + c, valid), y);
#pragma unroll
                for (int j = 0; j < kWide; ++j) {
                    d += (double)s[j] * (double)s[j];
                    e += (double)y[j] * (double)g[j] * (double)s[j];
                }
            }
            d = sum_all<T>(d, between64);
            e = sum_all<T>(e, between642);
            const double r64 = 1.0 / sqrt(d / (double)a.cols + (double)a.eps);
            r = split(r64);
            mean = (float)(e * r64 / (double)a.cols);
        }
#pragma unroll kUnroll
        for (int i = 0; i < (V ? V : pieces); ++i) {
            const int c = (i * T + lane) * kWide, valid = a.cols - c;
            if (valid <= 0) continue;
            float s[kWide], y[kWide], g[kWide], o[kWide], u[kWide];
            piece(i, c, valid, s, y, g);
            widen<BF>(V ? d8[V ? i : 0] : a.ds ? load8(dp + c, valid) : u32x4{0u, 0u, 0u, 0u}, o);
#pragma unroll
            for (int j = 0; j < kWide; ++j) {
                u[j] = times(s[j], r);
                o[j] += times(y[j] * g[j] - u[j] * mean, r);
                u[j] *= y[j];
            }
            if (a.dx)
                store8(static_cast<uint16_t *>(a.dx) + row * a.lddx + c, narrow<BF>(o), valid);
            if (V) {
#pragma unroll
                for (int j = 0; j < kWide; ++j) dg[V ? i : 0][j] += u[j];
            } else if (part) {
                for (int j = 0; j < kWide && j < valid; ++j)
                    part[c + j] = first ? u[j] : part[c + j] + u[j];
            }
        }
        first = false;
    }
    if (!V || !part) return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = (i * T + lane) * kWide, valid = a.cols - c;
        if (valid >= kWide) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<f32x4u *>(part + c + 4 * h) =
                    f32x4{dg[i][4 * h], dg[i][4 * h + 1], dg[i][4 * h + 2], dg[i][4 * h + 3]};
        } else {
#pragma unroll
            for (int j = 0; j < kWide; ++j)
                if (j < valid) part[c + j] = dg[i][j];
        }
    }
}

// dgain: the parts of 32 columns by a workgroup, eight lanes a part and 128 parts at a time, whose
// sums are added in two stages; always in the same order.
template <bool BF, bool G32>
__global__ void __launch_bounds__(1024)
gain_sum_kernel(const float *__restrict__ part, int parts, int cols, void *__restrict__ dgain) {
    __shared__ float between[128][33], again[8][32];
    const int set = threadIdx.x >> 3, c4 = (threadIdx.x & 7) * 4, c = blockIdx.x * 32 + c4;
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c + 4 <= cols)
        for (int p = set; p < parts; p += 128)
            sum += *reinterpret_cast<const f32x4u *>(part + (int64_t)p * cols + c);
    else
        for (int p = set; p < parts; p += 128)
            for (int i = 0; i < cols - c; ++i) sum[i] += part[(int64_t)p * cols + c + i];
#pragma unroll
    for (int i = 0; i < 4; ++i) between[set][c4 + i] = sum[i];
    __syncthreads();
    const int col = threadIdx.x & 31, sixteen = threadIdx.x >> 5;
    if (sixteen < 8) {
        float v = between[16 * sixteen][col];
#pragma unroll
        for (int i = 1; i < 16; ++i) v += between[16 * sixteen + i][col];
        again[sixteen][col] = v;
    }
    __syncthreads();
    if (threadIdx.x >= 32 || (int)blockIdx.x * 32 + col >= cols) return;
    float v = again[0][col];
#pragma unroll
    for (int i = 1; i < 8; ++i) v += again[i][col];
    if (G32)
        static_cast<float *>(dgain)[blockIdx.x * 32 + col] = v;
    else
        static_cast<uint16_t *>(dgain)[blockIdx.x * 32 + col] = Act<BF>::store(v);
}

// ---- blocks ----
// Activations: a lane takes 16 columns and eight lanes a block, so that a wave writes 1 KiB at a
// time.  A workgroup takes 2^(8 - shift) rows of up to 4,096 columns.  4,096 x 12,288: 28.7 us, 5.3
// TB/s; 8,200 x 2,048: 11.2 (12.9 with eight columns a lane and a division for the row).
template <bool BF>
__global__ void __launch_bounds__(256)
block_quantize_kernel(const uint16_t *__restrict__ x, int64_t ldx, int64_t n, int cols, int shift,
                      BlockRowsArgs q) {
    const int64_t row = ((int64_t)blockIdx.x << (8 - shift)) + (threadIdx.x >> shift);
    const int c = (int)((blockIdx.y << shift) + (threadIdx.x & ((1 << shift) - 1))) * 16;
    if (row >= n || c >= blocks_of(cols) * kBlock) return;    // whole blocks' lanes
    const uint16_t *at = x + row * ldx + c;
    float f[2][kWide];
    widen<BF>(load8(at, cols - c), f[0]);
    widen<BF>(load8(at + kWide, cols - c - kWide), f[1]);
    uint32_t big = larger(largest8(f[0]), largest8(f[1]));
    float v = __builtin_bit_cast(float, big);
    big = larger(big, __builtin_bit_cast(uint32_t, lane_xor<1>(v)));
    v = __builtin_bit_cast(float, big);
    big = larger(big, __builtin_bit_cast(uint32_t, lane_xor<2>(v)));
    v = __builtin_bit_cast(float, big);
    big = larger(big, __builtin_bit_cast(uint32_t, lane_xor<4>(v)));
    const CodeScale s = code_scale(big);
    const u32x2 lo = first_codes(to_codes(f[0], s), cols - c);
    const u32x2 hi = first_codes(to_codes(f[1], s), cols - c - kWide);
    *reinterpret_cast<u32x4 *>(q.q + row * q.ld + c) = u32x4{lo[0], lo[1], hi[0], hi[1]};
    if ((c & (kBlock - 1)) == 0) q.scale[(c / kBlock) * q.lds + row] = s.scale;
}

// A block of 128 x 128 of a matrix: 16 lanes of eight columns a row, 16 rows at a time, all held
// until the largest is known.  12,288 x 4,096, bfloat16: 27.4 us, 5.5 TB/s.
template <int TYPE>
__global__ void __launch_bounds__(256)
block_quantize_weight_kernel(const void *__restrict__ w, int64_t ldw, int rows, int cols,
                             uint8_t *__restrict__ q, int64_t ldq, float *__restrict__ scale) {
    __shared__ uint32_t wave_big[4];
    const int c = blockIdx.x * kBlock + (threadIdx.x & 15) * kWide, valid = cols - c;
    const int64_t r0 = (int64_t)blockIdx.y * kBlock + (threadIdx.x >> 4);
    float f[8][kWide];
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = r0 + 16 * i;
        const int there = row < rows ? valid : 0;
        if (TYPE == EXL3_F32)
            load_gain<false, true>(static_cast<const float *>(w) + (row < rows ? row : 0) * ldw, c,
                                   there, f[i]);
        else
            widen<TYPE == EXL3_BF16>(
                load8(static_cast<const uint16_t *>(w) + (row < rows ? row : 0) * ldw + c, there),
                f[i]);
        big = larger(big, largest8(f[i]));
    }
    for (int m = 1; m < 64; m <<= 1) big = larger(big, (uint32_t)__shfl_xor((int)big, m));
    if ((threadIdx.x & 63) == 0) wave_big[threadIdx.x >> 6] = big;
    __syncthreads();
    big = larger(larger(wave_big[0], wave_big[1]), larger(wave_big[2], wave_big[3]));
    const CodeScale s = code_scale(big);
    if (threadIdx.x == 0) scale[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = s.scale;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = r0 + 16 * i;
        if (row < rows)
            *reinterpret_cast<u32x2 *>(q + row * ldq + c) = first_codes(to_codes(f[i], s), valid);
    }
}

template <int T, int V, bool BF, bool G32>
hipError_t norm_t(const NormArgs &a, hipStream_t stream) {
    constexpr int kRows = T < 256 ? 256 / T : 1;
    NormArgs p = a;
    // rows a launch: a grid's side has fewer than 2^32 lanes
    const int64_t per = rows_a_launch(T < 256 ? 256 : T) * kRows;
    for (int64_t r0 = 0; r0 < a.n; r0 += per) {
        p.n = a.n - r0 < per ? a.n - r0 : per;
        p.x = static_cast<const uint16_t *>(a.x) + r0 * a.ldx;
        if (a.residual) p.residual = static_cast<const uint16_t *>(a.residual) + r0 * a.ldr;
        if (a.y) p.y = static_cast<uint16_t *>(a.y) + r0 * a.ldy;
        if (a.sum) p.sum = static_cast<uint16_t *>(a.sum) + r0 * a.ldsum;
        if (!a.y) {
            p.q.q = a.q.q + r0 * a.q.ld;
            p.q.scale = a.q.scale + r0;
        }
        hipLaunchKernelGGL((rms_norm_kernel<T, V, BF, G32>),
                           dim3((unsigned)((p.n + kRows - 1) / kRows)), dim3(T < 256 ? 256 : T), 0,
                           stream, p);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

template <bool BF, bool G32>
hipError_t norm_v(const NormArgs &a, hipStream_t stream) {
    if (a.cols <= 512) return norm_t<64, 1, BF, G32>(a, stream);
    if (a.cols <= 1024) return norm_t<64, 2, BF, G32>(a, stream);
    if (a.cols <= 2048) return norm_t<256, 1, BF, G32>(a, stream);
    if (a.cols <= 4096) return norm_t<512, 1, BF, G32>(a, stream);
    if (a.cols <= 8192) return norm_t<1024, 1, BF, G32>(a, stream);
    if (a.cols <= 16384) return norm_t<1024, 2, BF, G32>(a, stream);
    return norm_t<1024, 0, BF, G32>(a, stream);
}

template <bool BF, bool G32>
hipError_t backward_v(const NormBackwardArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)a.parts);
#define EXL3_BACK(T, V)                                                                       \
    hipLaunchKernelGGL((rms_norm_backward_kernel<T, V, BF, G32>), grid, dim3(T), 0, stream, a)
    if (a.n > 0) {
        if (a.cols <= 1024)
            EXL3_BACK(128, 1);
        else if (a.cols <= 2048)
            EXL3_BACK(256, 1);
        else if (a.cols <= 4096)
            EXL3_BACK(512, 1);
        else if (a.cols <= 8192)
            EXL3_BACK(512, 2);
        else if (a.cols <= 16384)
            EXL3_BACK(1024, 2);
        else
            EXL3_BACK(1024, 0);
    }
#undef EXL3_BACK
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || !a.dgain) return err;
    hipLaunchKernelGGL((gain_sum_kernel<BF, G32>), dim3((unsigned)((a.cols + 31) / 32)), dim3(1024),
                       0, stream, a.part, a.n > 0 ? a.parts : 0, a.cols, a.dgain);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs &a, bool bf16, hipStream_t stream) {
    if (bf16) return a.gain32 ? norm_v<true, true>(a, stream) : norm_v<true, false>(a, stream);
    return a.gain32 ? norm_v<false, true>(a, stream) : norm_v<false, false>(a, stream);
}

// Workgroups, each with a part of dgain, that write 4 bytes a column more.  A compute unit's, us:
// 2,000 x 4,096: one 22.9, two 19.8, three 22.4; 4,000 x 1,000: one 29, two 21, four 17.4;
// 2,000 x 8,192: one 39, two 42.
int norm_backward_parts(int64_t n, int cols, int n_cu) {
    const int64_t most = (int64_t)n_cu * (cols <= 1024 ? 4 : cols <= 2048 ? 3 : cols <= 4096 ? 2 : 1);
    return (int)(n < most ? n : most);
}

hipError_t launch_rms_norm_backward(const NormBackwardArgs &a, bool bf16, hipStream_t stream) {
    if (bf16)
        return a.gain32 ? backward_v<true, true>(a, stream) : backward_v<true, false>(a, stream);
    return a.gain32 ? backward_v<false, true>(a, stream) : backward_v<false, false>(a, stream);
}

hipError_t launch_block_quantize(const void *x, int64_t ldx, int64_t n, int cols, bool bf16,
                                 const BlockRowsArgs &out, hipStream_t stream) {
    const int pieces = blocks_of(cols) * (kBlock / 16);
    int shift = 3;                               // lanes a row, a power of two
    while (shift < 8 && (1 << shift) < pieces) ++shift;
    const unsigned across = (unsigned)((pieces + (1 << shift) - 1) >> shift);
    const int64_t per = rows_a_launch(256) << (8 - shift);
    for (int64_t r0 = 0; r0 < n; r0 += per) {
        const int64_t rows = n - r0 < per ? n - r0 : per;
        const dim3 grid((unsigned)((rows + (256 >> shift) - 1) >> (8 - shift)), across);
        const uint16_t *xx = static_cast<const uint16_t *>(x) + r0 * ldx;
        const BlockRowsArgs q{out.q + r0 * out.ld, out.scale + r0, out.ld, out.lds};
        if (bf16)
            hipLaunchKernelGGL((block_quantize_kernel<true>), grid, dim3(256), 0, stream, xx, ldx,
                               rows, cols, shift, q);
        else
            hipLaunchKernelGGL((block_quantize_kernel<false>), grid, dim3(256), 0, stream, xx, ldx,
                               rows, cols, shift, q);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

hipError_t launch_block_quantize_weight(const void *w, int dtype, int64_t ldw, int rows, int cols,
                                        uint8_t *q, int64_t ldq, float *scale, hipStream_t stream) {
    const dim3 grid((unsigned)blocks_of(cols), (unsigned)blocks_of(rows));
#define EXL3_WEIGHT(TYPE)                                                                       \
    hipLaunchKernelGGL((block_quantize_weight_kernel<TYPE>), grid, dim3(256), 0, stream, w, ldw, \
                       rows, cols, q, ldq, scale)
    if (dtype == EXL3_F32)
        EXL3_WEIGHT(EXL3_F32);
    else if (dtype == EXL3_BF16)
        EXL3_WEIGHT(EXL3_BF16);
    else
        EXL3_WEIGHT(EXL3_F16);
#undef EXL3_WEIGHT
    return hipGetLastError();
}

}  // namespace exl3
