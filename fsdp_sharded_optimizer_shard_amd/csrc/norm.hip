// Layer norm, forward and backward, with the sums of the gain's and the bias's
// gradients.
//
// With n columns, mu = sum x / n, var = sum (x - mu)^2 / n, r = 1 / sqrt(var + eps)
// and xh = (x - mu) r:
//   y  = xh g + b
//   h  = dy g
//   dx = r (h - sum(h) / n - xh sum(h xh) / n)  [+ residual]
//   dg = sum over rows of dy xh,   db = sum over rows of dy.
// Nothing here is a product of matrices: each row is read once, held in
// registers over its sums, and written once, so memory bounds it.  The variance
// is summed about the mean from the held row, not as a difference of squares.
// All sums are fp32 in a fixed order.
#include <hip/hip_runtime.h>

#include "checks.h"
#include "vec.h"

namespace zs {
namespace {

// Eight neighbouring values as loaded: bf16 in w[0], fp32 in both (W: fp32 is
// possible).
template <bool W>
struct Raw8 {
    uint4 w[W ? 2 : 1];
};

template <bool W>
__device__ __forceinline__ Raw8<W> raw8(const void *p, bool bf16, int64_t i, int n)
{
    Raw8<W> r = {};
    if (n <= 0)
        return r;
    if (n == 8) {
        if (!W || bf16) {
            r.w[0] = load16(static_cast<const uint16_t *>(p) + i);
        } else {
            r.w[0] = load16(static_cast<const float *>(p) + i);
            r.w[W ? 1 : 0] = load16(static_cast<const float *>(p) + i + 4);
        }
        return r;
    }
    uint32_t w[8] = {};
    if (!W || bf16) {
        const uint16_t *q = static_cast<const uint16_t *>(p) + i;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n)
                w[k >> 1] |= (uint32_t)q[k] << (16 * (k & 1));
    } else {
        const uint32_t *q = static_cast<const uint32_t *>(p) + i;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n)
                w[k] = q[k];
    }
    r.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
    if constexpr (W)
        r.w[1] = make_uint4(w[4], w[5], w[6], w[7]);
    return r;
}

template <bool W>
__device__ __forceinline__ void unraw8(const Raw8<W> &r, bool bf16, float (&x)[8])
{
    if (!W || bf16) {
        widen8(r.w[0], x);
    } else if constexpr (W) {
        const uint32_t w[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
        for (int k = 0; k < 8; ++k)
            x[k] = __uint_as_float(w[k]);
    }
}

__device__ __forceinline__ float wave_sum(float x)
{
#pragma unroll
    for (int s = 1; s < 64; s *= 2)
        x += __shfl_xor(x, s, 64);
    return x;
}

// Sums of two values over the TPR threads of a row, the same in each of them.
// `slot`: 2 x 16 floats of LDS of this row's group; every thread of the block
// has to come.
template <int TPR>
__device__ __forceinline__ void row_sums(float &a, float &b, float *slot)
{
    a = wave_sum(a);
    b = wave_sum(b);
    if constexpr (TPR > 64) {
        const int w = (threadIdx.x % TPR) >> 6;
        if ((threadIdx.x & 63) == 0) {
            slot[w] = a;
            slot[16 + w] = b;
        }
        __syncthreads();
        a = slot[0];
        b = slot[16];
#pragma unroll
        for (int i = 1; i < TPR / 64; ++i) {
            a += slot[i];
            b += slot[16 + i];
        }
    }
}

struct NormArgs {
    int64_t rows, cols;
    const void *x;
    int64_t ldx;
    const void *gain, *bias;
    void *y;
    int64_t ldy;
    float *mean, *rstd;
    float eps, inv_n;
    bool x_bf16, p_bf16, y_bf16;
};

// TPR threads a row, each NC chunks of eight columns, TPR chunks apart.  A block of
// THREADS takes rows blockIdx.x, + gridDim.x, ... of groups of THREADS / TPR rows: the
// gain and the bias stay in registers, and the next row's loads go out before the
// present one's sums meet.
template <int THREADS, int TPR, int NC, bool W>
__global__ __launch_bounds__(THREADS) void norm_forward_kernel(const NormArgs p)
{
    constexpr int RPB = THREADS / TPR;
    __shared__ float slots[2][2][RPB][32];
    const int t = threadIdx.x % TPR, g = threadIdx.x / TPR;
    const int64_t step = (int64_t)gridDim.x * RPB;
    Raw8<W> raw[NC], rg[NC], rb[NC];
    int n[NC];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < NC; ++j)
            raw[j] = raw8<W>(p.x, p.x_bf16, row * p.ldx + (int64_t)(t + j * TPR) * 8, row < p.rows ? n[j] : 0);
    };
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        const int64_t left = p.cols - (int64_t)(t + j * TPR) * 8;
        n[j] = left < 0 ? 0 : left < 8 ? (int)left : 8;
    }
    fetch((int64_t)blockIdx.x * RPB + g);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        const int64_t col = (int64_t)(t + j * TPR) * 8;
        rg[j] = raw8<W>(p.gain, p.p_bf16, col, p.gain ? n[j] : 0);
        rb[j] = raw8<W>(p.bias, p.p_bf16, col, p.bias ? n[j] : 0);
    }
    int turn = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < p.rows; row0 += step, turn ^= 1) {
        const int64_t row = row0 + g;
        const bool here = row < p.rows;
        float x[NC][8], s = 0.0f, q = 0.0f, none = 0.0f;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            unraw8(raw[j], p.x_bf16, x[j]);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                s += x[j][k];
        }
        fetch(row + step);
        row_sums<TPR>(s, none, slots[turn][0][g]);
        const float mu = s * p.inv_n;
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                x[j][k] -= mu;
                q += k < n[j] ? x[j][k] * x[j][k] : 0.0f;
            }
        row_sums<TPR>(q, none, slots[turn][1][g]);
        const float r = 1.0f / sqrtf(q * p.inv_n + p.eps);
        if (here && t == 0) {
            if (p.mean)
                p.mean[row] = mu;
            if (p.rstd)
                p.rstd[row] = r;
        }
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            if (!here || n[j] == 0)
                break;
            float gain[8], bias[8];
            unraw8(rg[j], p.p_bf16, gain);
            unraw8(rb[j], p.p_bf16, bias);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[j][k] = __builtin_fmaf(x[j][k] * r, p.gain ? gain[k] : 1.0f, bias[k]);
            store8(p.y, p.y_bf16, row * p.ldy + (int64_t)(t + j * TPR) * 8, n[j] == 8, n[j], x[j]);
        }
    }
}

// Rows too long to be held: read three times, the second and third time from
// the caches.
__global__ __launch_bounds__(1024) void norm_forward_long_kernel(const NormArgs p)
{
    __shared__ float slots[2][32];
    const int64_t row = blockIdx.x, at = row * p.ldx;
    float s = 0.0f, q = 0.0f, none = 0.0f, x[8];
    auto each = [&](auto f) {
        for (int64_t col = (int64_t)threadIdx.x * 8; col < p.cols; col += 8192) {
            const int n = (int)(p.cols - col < 8 ? p.cols - col : 8);
            unraw8(raw8<true>(p.x, p.x_bf16, at + col, n), p.x_bf16, x);
            f(col, n);
        }
    };
    each([&](int64_t, int) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            s += x[k];
    });
    row_sums<1024>(s, none, slots[0]);
    const float mu = s * p.inv_n;
    each([&](int64_t, int n) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            q += k < n ? (x[k] - mu) * (x[k] - mu) : 0.0f;
    });
    row_sums<1024>(q, none, slots[1]);
    const float r = 1.0f / sqrtf(q * p.inv_n + p.eps);
    if (threadIdx.x == 0) {
        if (p.mean)
            p.mean[row] = mu;
        if (p.rstd)
            p.rstd[row] = r;
    }
    each([&](int64_t col, int n) {
        float gain[8], bias[8];
        unraw8(raw8<true>(p.gain, p.p_bf16, col, p.gain ? n : 0), p.p_bf16, gain);
        unraw8(raw8<true>(p.bias, p.p_bf16, col, p.bias ? n : 0), p.p_bf16, bias);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            x[k] = __builtin_fmaf((x[k] - mu) * r, p.gain ? gain[k] : 1.0f, bias[k]);
        store8(p.y, p.y_bf16, row * p.ldy + col, n == 8, n, x);
    });
}

struct NormBackArgs {
    int64_t rows, cols;
    const void *dy, *x, *gain, *res;
    int64_t ldy, ldx, ldr, ldd;
    const float *mean, *rstd;
    void *dx;
    float *dgain, *dbias;  // one row of sums a block: gridDim.x x cols each; NULL: left out
    float inv_n;
    bool y_bf16, x_bf16, p_bf16, d_bf16;
};

// A block of 1024 threads takes rows blockIdx.x, + gridDim.x, ... of groups of
// RPB rows, TPR threads a row; a thread keeps its columns' sums in registers
// over all of them, so that a block leaves one row of sums.  The next row's loads
// go out before the present one's sums meet, where a thread has one chunk.  With 1024
// threads a thread has 128 registers, of which bf16 rows of one chunk take 98 to 108.
// Two chunks do not fit, even without a second row: 24 to 26 values go to scratch.
// Operands in fp32 leave 6 or 7 there up to 4096 columns.  4096 rows of 8192 with a
// residual, 268 MB: 52 us, and 5 for the blocks' sums (a copy of as much: 46); all in
// fp32, 537 MB, 110 in all; 8192 rows of 4096 55 in bf16 and 112 in fp32.  A few long rows
// are bound by their blocks' rows of sums, written and read again: 181 of 14363, 37 us.
constexpr int kNormThreads = 1024;
constexpr int kNormBlocks = 256;  // one a CU; a fixed number, so that the sums have the same bits everywhere

template <int TPR, int NC, bool W>
__global__ __launch_bounds__(kNormThreads) void norm_backward_kernel(const NormBackArgs p)
{
    constexpr int RPB = kNormThreads / TPR;
    __shared__ float slots[2][RPB][32];
    __shared__ float part[RPB > 1 ? 8 * kNormThreads : 1];
    const int t = threadIdx.x % TPR, g = threadIdx.x / TPR;
    const int64_t step = (int64_t)gridDim.x * RPB;
    float sg[NC][8], sb[NC][8];
    Raw8<W> ry[NC], rx[NC], rr[NC];
    int n[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        const int64_t left = p.cols - (int64_t)(t + j * TPR) * 8;
        n[j] = left < 0 ? 0 : left < 8 ? (int)left : 8;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            sg[j][k] = sb[j][k] = 0.0f;
    }
    float mu = 0.0f, r = 0.0f;
    auto fetch = [&](int64_t row) {
        const bool here = row < p.rows;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            const int64_t col = (int64_t)(t + j * TPR) * 8;
            const int m = here ? n[j] : 0;
            ry[j] = raw8<W>(p.dy, p.y_bf16, row * p.ldy + col, m);
            rx[j] = raw8<W>(p.x, p.x_bf16, row * p.ldx + col, m);
            rr[j] = raw8<W>(p.res, p.d_bf16, row * p.ldr + col, p.res ? m : 0);
        }
        mu = here ? p.mean[row] : 0.0f;
        r = here ? p.rstd[row] : 0.0f;
    };
    fetch((int64_t)blockIdx.x * RPB + g);
    int turn = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < p.rows; row0 += step, turn ^= 1) {
        const int64_t row = row0 + g;
        const bool here = row < p.rows;
        float xh[NC][8], h[NC][8], res[NC][8], s1 = 0.0f, s2 = 0.0f;
        const float rs = r;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            float dy[8], gain[8];
            unraw8(ry[j], p.y_bf16, dy);
            unraw8(rx[j], p.x_bf16, xh[j]);
            unraw8(rr[j], p.d_bf16, res[j]);
            unraw8(raw8<true>(p.gain, p.p_bf16, (int64_t)(t + j * TPR) * 8, p.gain ? n[j] : 0), p.p_bf16,
                   gain);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                xh[j][k] = k < n[j] ? (xh[j][k] - mu) * r : 0.0f;
                h[j][k] = p.gain ? dy[k] * gain[k] : dy[k];
                sb[j][k] += dy[k];
                sg[j][k] = __builtin_fmaf(dy[k], xh[j][k], sg[j][k]);
                s1 += h[j][k];
                s2 = __builtin_fmaf(h[j][k], xh[j][k], s2);
            }
        }
        if constexpr (NC == 1)
            fetch(row + step);
        row_sums<TPR>(s1, s2, slots[turn][g]);
        s1 *= p.inv_n;
        s2 *= p.inv_n;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            if (!here || n[j] == 0)
                break;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                h[j][k] = __builtin_fmaf(rs, __builtin_fmaf(-xh[j][k], s2, h[j][k] - s1), res[j][k]);
            store8(p.dx, p.d_bf16, row * p.ldd + (int64_t)(t + j * TPR) * 8, n[j] == 8, n[j], h[j]);
        }
        if constexpr (NC > 1)
            fetch(row + step);
    }
    // The groups' sums, added in order by the first.
    auto leave = [&](float (&s)[NC][8], float *out) {
        if (!out)
            return;
        out += (int64_t)blockIdx.x * p.cols;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            if constexpr (RPB > 1) {
                __syncthreads();
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    part[k * kNormThreads + threadIdx.x] = s[j][k];
                __syncthreads();
                if (g == 0)
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        for (int i = 1; i < RPB; ++i)
                            s[j][k] += part[k * kNormThreads + i * TPR + t];
            }
            if (g == 0)
                store8(out, false, (int64_t)(t + j * TPR) * 8,
                       n[j] == 8 && (reinterpret_cast<uintptr_t>(out) & 15) == 0, n[j], s[j]);
        }
    };
    leave(sg, p.dgain);
    leave(sb, p.dbias);
}

// Rows too long to be held: the row's sums in one pass, then dx in another; the
// columns' sums by a kernel of their own.
__global__ __launch_bounds__(1024) void norm_backward_long_kernel(const NormBackArgs p)
{
    __shared__ float slots[32];
    const int64_t row = blockIdx.x;
    const float mu = p.mean[row], r = p.rstd[row];
    float s1 = 0.0f, s2 = 0.0f, h[8], xh[8];
    auto each = [&](auto f) {
        for (int64_t col = (int64_t)threadIdx.x * 8; col < p.cols; col += 8192) {
            const int n = (int)(p.cols - col < 8 ? p.cols - col : 8);
            float gain[8];
            unraw8(raw8<true>(p.dy, p.y_bf16, row * p.ldy + col, n), p.y_bf16, h);
            unraw8(raw8<true>(p.x, p.x_bf16, row * p.ldx + col, n), p.x_bf16, xh);
            unraw8(raw8<true>(p.gain, p.p_bf16, col, p.gain ? n : 0), p.p_bf16, gain);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                xh[k] = k < n ? (xh[k] - mu) * r : 0.0f;
                h[k] = p.gain ? h[k] * gain[k] : h[k];
            }
            f(col, n);
        }
    };
    each([&](int64_t, int) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            s1 += h[k];
            s2 = __builtin_fmaf(h[k], xh[k], s2);
        }
    });
    row_sums<1024>(s1, s2, slots);
    s1 *= p.inv_n;
    s2 *= p.inv_n;
    each([&](int64_t col, int n) {
        float res[8];
        unraw8(raw8<true>(p.res, p.d_bf16, row * p.ldr + col, p.res ? n : 0), p.d_bf16, res);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            h[k] = __builtin_fmaf(r, __builtin_fmaf(-xh[k], s2, h[k] - s1), res[k]);
        store8(p.dx, p.d_bf16, row * p.ldd + col, n == 8, n, h);
    });
}

// Column sums of dy xh and dy alone, before dx may overwrite dy: a block takes
// 512 columns of the rows blockIdx.y, + gridDim.y, ...
__global__ __launch_bounds__(64) void norm_columns_kernel(const NormBackArgs p)
{
    const int64_t col = (int64_t)blockIdx.x * 512 + threadIdx.x * 8;
    const int64_t left = p.cols - col;
    if (left <= 0)
        return;
    const int n = left < 8 ? (int)left : 8;
    float sg[8] = {}, sb[8] = {};
    for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
        const float mu = p.mean[row], r = p.rstd[row];
        float dy[8], x[8];
        unraw8(raw8<true>(p.dy, p.y_bf16, row * p.ldy + col, n), p.y_bf16, dy);
        unraw8(raw8<true>(p.x, p.x_bf16, row * p.ldx + col, n), p.x_bf16, x);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            sb[k] += dy[k];
            sg[k] = __builtin_fmaf(dy[k], (x[k] - mu) * r, sg[k]);
        }
    }
    const int64_t at = (int64_t)blockIdx.y * p.cols + col;
    if (p.dgain)
        store8(p.dgain, false, at, n == 8, n, sg);
    if (p.dbias)
        store8(p.dbias, false, at, n == 8, n, sb);
}

// out[c] = sum of n rows of partial sums, for one or two outputs (blockIdx.y):
// 32 columns a block, its 32 half waves a 32nd of the rows each, added in order.
__global__ __launch_bounds__(1024) void norm_sum_kernel(const float *__restrict__ pg, const float *__restrict__ pb,
                                                        int n, int64_t cols, float *__restrict__ dgain,
                                                        float *__restrict__ dbias)
{
    __shared__ float part[32][33];
    const float *in = blockIdx.y ? pb : pg;
    float *out = blockIdx.y ? dbias : dgain;
    const int c = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int64_t col = (int64_t)blockIdx.x * 32 + c;
    float s = 0.0f;
    if (out && col < cols) {
#pragma unroll 8
        for (int i = q; i < n; i += 32)
            s += in[(int64_t)i * cols + col];
    }
    part[q][c] = s;
    __syncthreads();
    if (q == 0 && out && col < cols) {
#pragma unroll
        for (int i = 1; i < 32; ++i)
            s += part[i][c];
        out[col] = s;
    }
}

__global__ __launch_bounds__(256) void fill_zero_kernel(float *p, int64_t n)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        p[i] = 0.0f;
}

constexpr int64_t kHeld = 16384;  // the longest row that is held in registers
// Rows: held ones are strided over; of the longer ones each takes a block of 1024, and
// the dispatch counts threads in 32 bits.
constexpr int64_t kMaxRows = 0x7fffffff, kMaxLongRows = int64_t(0xffffffffu) / 1024;
// Columns that norm_sum_kernel's blocks of 1024 threads have, 32 each.
constexpr int64_t kMaxSumCols = int64_t(0xffffffffu) / 1024 * 32;

// Threads a row of the backward kernel: eight columns each up to 8192.
int back_tpr(int64_t cols)
{
    int t = 64;
    while (t < kNormThreads && cols > 8 * t)
        t *= 2;
    return t;
}

// Rows of partial sums, 0: the kernel writes the sums themselves.
int64_t norm_blocks(int64_t rows, int64_t cols)
{
    if (cols > kHeld)
        return rows < kNormBlocks ? rows : kNormBlocks;
    const int64_t rpb = kNormThreads / back_tpr(cols), b = (rows + rpb - 1) / rpb;
    return b < kNormBlocks ? b : kNormBlocks;
}

zero_status norm_common(int64_t rows, int64_t cols, const void *x, int64_t ldx, int32_t x_dtype,
                        const void *gain, const void *bias, int32_t param_dtype)
{
    zero_status st;
    if ((st = check_extent(rows, cols, ldx)) != ZERO_OK)
        return st;
    if (!known_dtype(x_dtype) || !known_dtype(param_dtype))
        return fail(ZERO_ERR_INVALID_ARG, "unknown dtype (x %d, parameters %d)", x_dtype, param_dtype);
    if (rows > (cols > kHeld ? kMaxLongRows : kMaxRows))
        return fail(ZERO_ERR_UNSUPPORTED, "%lld rows of %lld columns are too many for one launch", (long long)rows,
                    (long long)cols);
    if (!aligned(gain, bytes_of(param_dtype)) || !aligned(bias, bytes_of(param_dtype)))
        return fail(ZERO_ERR_ALIGNMENT, "gain and bias must be aligned to their type");
    if (rows == 0 || cols == 0)
        return ZERO_OK;
    return check_matrix("x", x, ldx, cols, x_dtype);
}


}  // namespace
}  // namespace zs

extern "C" {

zero_status zero_layer_norm_forward(int64_t rows, int64_t cols, const void *x, int64_t ldx, int32_t x_dtype,
                                    const void *gain, const void *bias, int32_t param_dtype, float eps,
                                    void *y, int64_t ldy, int32_t y_dtype, float *mean, float *rstd,
                                    void *stream)
{
    using namespace zs;
    zero_status st;
    if ((st = norm_common(rows, cols, x, ldx, x_dtype, gain, bias, param_dtype)) != ZERO_OK ||
        (st = check_extent(rows, cols, ldy)) != ZERO_OK)
        return st;
    if (!known_dtype(y_dtype))
        return fail(ZERO_ERR_INVALID_ARG, "y: unknown dtype %d", y_dtype);
    if (!(eps >= 0.0f))
        return fail(ZERO_ERR_INVALID_ARG, "eps must not be negative");
    if (!aligned(mean, 4) || !aligned(rstd, 4))
        return fail(ZERO_ERR_ALIGNMENT, "mean and rstd must be 4-byte aligned");
    if (rows == 0 || cols == 0)
        return ZERO_OK;
    if ((st = check_matrix("y", y, ldy, cols, y_dtype)) != ZERO_OK)
        return st;
    if (y == x && (y_dtype != x_dtype || ldy != ldx))
        return fail(ZERO_ERR_INVALID_ARG, "y in place of x needs its type and leading dimension");
    if (is_one_of(y, {gain, bias, mean, rstd}) || is_one_of(mean, {x, gain, bias, rstd}) ||
        is_one_of(rstd, {x, gain, bias}))
        return fail(ZERO_ERR_INVALID_ARG, "y, mean and rstd need memory apart from what the call reads and "
                    "from each other");
    NormArgs p = {};
    p.rows = rows, p.cols = cols;
    p.x = x, p.ldx = ldx, p.gain = gain, p.bias = bias, p.y = y, p.ldy = ldy;
    p.mean = mean, p.rstd = rstd, p.eps = eps, p.inv_n = (float)(1.0 / (double)cols);
    p.x_bf16 = x_dtype == ZERO_BF16, p.p_bf16 = param_dtype == ZERO_BF16, p.y_bf16 = y_dtype == ZERO_BF16;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
#define ZS_NORM(THREADS, TPR, NC)                                                                  \
    do {                                                                                           \
        const int64_t groups = (rows + THREADS / TPR - 1) / (THREADS / TPR);                       \
        const dim3 grid((unsigned)(groups < most / THREADS ? groups : most / THREADS));            \
        if (wide)                                                                                  \
            hipLaunchKernelGGL((norm_forward_kernel<THREADS, TPR, NC, true>), grid, dim3(THREADS), 0, s, p); \
        else                                                                                       \
            hipLaunchKernelGGL((norm_forward_kernel<THREADS, TPR, NC, false>), grid, dim3(THREADS), 0, s, p); \
    } while (0)
    const bool wide = !(p.x_bf16 && p.p_bf16);
    // Two chunks a thread and 1024 threads a CU: 128 MB through rows of 8192 in 27 us
    // (a copy: 26.5), one chunk a thread 44, four 31; twice the threads 29 to 32.  Rows
    // of up to 512, of one chunk, take 27.6 us with 2048 threads a CU and 33 with 1024.
    const int64_t most = (cols <= 512 ? 512 : 256) * 1024;
    if (cols <= 512)
        ZS_NORM(256, 64, 1);
    else if (cols <= 1024)
        ZS_NORM(256, 64, 2);
    else if (cols <= 2048)
        ZS_NORM(256, 128, 2);
    else if (cols <= 4096)
        ZS_NORM(256, 256, 2);
    else if (cols <= 8192)
        ZS_NORM(512, 512, 2);
    else if (cols <= kHeld)
        ZS_NORM(1024, 1024, 2);
    else
        hipLaunchKernelGGL(norm_forward_long_kernel, dim3((unsigned)rows), dim3(1024), 0, s, p);
#undef ZS_NORM
    return launched("layer_norm_forward");
}

int64_t zero_layer_norm_workspace(int64_t rows, int64_t cols)
{
    if (rows <= 0 || cols <= 0)
        return 0;
    const int64_t b = zs::norm_blocks(rows, cols);
    return b > 1 ? 2 * b * cols : 0;
}

zero_status zero_layer_norm_backward(int64_t rows, int64_t cols, const void *dy, int64_t lddy, int32_t dy_dtype,
                                     const void *x, int64_t ldx, int32_t x_dtype, const void *gain,
                                     int32_t param_dtype, const float *mean, const float *rstd,
                                     const void *residual, int64_t ldr, void *dx, int64_t lddx,
                                     int32_t dx_dtype, float *dgain, float *dbias, float *workspace,
                                     int64_t n_workspace, void *stream)
{
    using namespace zs;
    zero_status st;
    if ((st = norm_common(rows, cols, x, ldx, x_dtype, gain, nullptr, param_dtype)) != ZERO_OK ||
        (st = check_extent(rows, cols, lddy)) != ZERO_OK || (st = check_extent(rows, cols, lddx)) != ZERO_OK ||
        (residual && (st = check_extent(rows, cols, ldr)) != ZERO_OK))
        return st;
    if (!known_dtype(dy_dtype) || !known_dtype(dx_dtype))
        return fail(ZERO_ERR_INVALID_ARG, "unknown dtype (dy %d, dx %d)", dy_dtype, dx_dtype);
    for (const void *f : {(const void *)mean, (const void *)rstd, (const void *)dgain, (const void *)dbias,
                          (const void *)workspace})
        if (!aligned(f, 4))
            return fail(ZERO_ERR_ALIGNMENT, "mean, rstd, dgain, dbias and workspace must be 4-byte aligned");
    if (cols == 0)
        return ZERO_OK;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (rows == 0) {
        if (dgain && dgain == dbias)
            return fail(ZERO_ERR_INVALID_ARG, "dgain and dbias need memory each");
        for (float *f : {dgain, dbias})
            if (f) {
                int64_t grid = (cols + 255) / 256;
                grid = grid > 65536 ? 65536 : grid;
                (void)hipGetLastError();
                hipLaunchKernelGGL(fill_zero_kernel, dim3((unsigned)grid), dim3(256), 0, s, f, cols);
                if ((st = launched("layer_norm_backward")) != ZERO_OK)
                    return st;
            }
        return ZERO_OK;
    }
    if ((st = check_matrix("dy", dy, lddy, cols, dy_dtype)) != ZERO_OK ||
        (st = check_matrix("dx", dx, lddx, cols, dx_dtype)) != ZERO_OK ||
        (residual && (st = check_matrix("residual", residual, ldr, cols, dx_dtype)) != ZERO_OK))
        return st;
    if (!mean || !rstd)
        return fail(ZERO_ERR_INVALID_ARG, "mean and rstd of the forward pass are required");
    if ((dx == dy && (dx_dtype != dy_dtype || lddx != lddy)) || (dx == x && (dx_dtype != x_dtype || lddx != ldx)) ||
        (dx == residual && lddx != ldr))
        return fail(ZERO_ERR_INVALID_ARG, "dx in place of another matrix needs its type and leading dimension");
    const int64_t need = dgain || dbias ? zero_layer_norm_workspace(rows, cols) : 0;
    if (need > 0 && cols > kMaxSumCols)
        return fail(ZERO_ERR_UNSUPPORTED, "dgain and dbias: %lld columns are too many for one launch", (long long)cols);
    if (need > 0 && (!workspace || n_workspace < need))
        return fail(ZERO_ERR_INVALID_ARG, "dgain and dbias of %lld x %lld need a workspace of %lld floats",
                    (long long)rows, (long long)cols, (long long)need);
    const void *w = need > 0 ? workspace : nullptr;
    if (is_one_of(dx, {gain, mean, rstd, dgain, dbias, w}) ||
        is_one_of(dgain, {dy, x, gain, mean, rstd, residual, dbias, w}) ||
        is_one_of(dbias, {dy, x, gain, mean, rstd, residual, w}) ||
        is_one_of(w, {dy, x, gain, mean, rstd, residual}))
        return fail(ZERO_ERR_INVALID_ARG, "dx, dgain, dbias and the workspace need memory apart from what the "
                    "call reads and from each other");
    NormBackArgs p = {};
    p.rows = rows, p.cols = cols;
    p.dy = dy, p.x = x, p.gain = gain, p.res = residual;
    p.ldy = lddy, p.ldx = ldx, p.ldr = ldr, p.ldd = lddx;
    p.mean = mean, p.rstd = rstd, p.dx = dx, p.inv_n = (float)(1.0 / (double)cols);
    p.y_bf16 = dy_dtype == ZERO_BF16, p.x_bf16 = x_dtype == ZERO_BF16;
    p.p_bf16 = param_dtype == ZERO_BF16, p.d_bf16 = dx_dtype == ZERO_BF16;
    const int64_t blocks = norm_blocks(rows, cols);
    const bool direct = blocks <= 1;
    float *const pg = !dgain ? nullptr : direct ? dgain : workspace;
    float *const pb = !dbias ? nullptr : direct ? dbias : workspace + blocks * cols;
    p.dgain = pg, p.dbias = pb;
    (void)hipGetLastError();
#define ZS_NORM(TPR, NC)                                                                           \
    do {                                                                                           \
        if (wide)                                                                                  \
            hipLaunchKernelGGL((norm_backward_kernel<TPR, NC, true>), dim3((unsigned)blocks),      \
                               dim3(kNormThreads), 0, s, p);                                       \
        else                                                                                       \
            hipLaunchKernelGGL((norm_backward_kernel<TPR, NC, false>), dim3((unsigned)blocks),     \
                               dim3(kNormThreads), 0, s, p);                                       \
    } while (0)
    const bool wide = !(p.y_bf16 && p.x_bf16 && p.d_bf16);
    if (cols > kHeld) {
        if (dgain || dbias)
            hipLaunchKernelGGL(norm_columns_kernel, dim3((unsigned)((cols + 511) / 512), (unsigned)blocks), dim3(64),
                               0, s, p);
        hipLaunchKernelGGL(norm_backward_long_kernel, dim3((unsigned)rows), dim3(1024), 0, s, p);
    } else if (cols <= 512) {
        ZS_NORM(64, 1);
    } else if (cols <= 1024) {
        ZS_NORM(128, 1);
    } else if (cols <= 2048) {
        ZS_NORM(256, 1);
    } else if (cols <= 4096) {
        ZS_NORM(512, 1);
    } else if (cols <= 8192) {
        ZS_NORM(1024, 1);
    } else {
        ZS_NORM(1024, 2);
    }
#undef ZS_NORM
    if ((st = launched("layer_norm_backward")) != ZERO_OK || direct || !(dgain || dbias))
        return st;
    hipLaunchKernelGGL(norm_sum_kernel, dim3((unsigned)((cols + 31) / 32), 2), dim3(1024), 0, s, pg, pb, (int)blocks,
                       cols, dgain, dbias);
    return launched("layer_norm sums");
}

}  // extern "C"
