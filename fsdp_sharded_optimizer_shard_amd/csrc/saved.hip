// The elementwise layer operators: activations into 8 bits and back, and the
// gradient of a product's epilogue.  All of them are bound by memory.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "act.h"
#include "checks.h"
#include "products.h"
#include "vec.h"

namespace zs {
namespace {

// One wave: 32 rows x 128 columns, lane = 8 columns of 8 rows, so that a
// block's largest magnitude is 8 values in the lane and two exchanges, and
// every load is 16 bytes.  Reading back moves 3.03 bytes an element at 6.4 TB/s
// (27.6 us at 4096 x 14336).
struct Spot {
    int64_t block, row, col;
    int rg;
};

__device__ __forceinline__ Spot spot(int64_t wave, int64_t col_waves)
{
    const int lane = threadIdx.x & 63;
    Spot s;
    s.block = wave / col_waves;
    s.rg = lane >> 4;
    s.row = s.block * 32 + s.rg * 8;
    s.col = (wave % col_waves) * 128 + (lane & 15) * 8;
    return s;
}

// Eight neighbouring inputs as loaded: bf16 stays packed.
template <bool BF16>
struct Raw {
    uint32_t w[BF16 ? 4 : 8];
    __device__ __forceinline__ float at(int k) const
    {
        if (BF16)
            return __uint_as_float(k & 1 ? w[k >> 1] & 0xffff0000u : w[k >> 1] << 16);
        return __uint_as_float(w[k]);
    }
};

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// Writes a checkpoint.  The largest magnitude of a block is a maximum over
// bit patterns with the sign off -- in bf16 two at a time -- which is right
// as long as nothing in the wave's blocks needs the coder's bounds; where
// something reaches 0x7f70 (240 * 2^120, infinities, NaN), the wave takes the
// maximum again without what must not count and bounds each value.  Testing
// and bounding every value took 46 us at 4096 x 14336 where this takes 32 (5.6
// TB/s; 40 us, 4.4 TB/s, where the input comes from HBM every time).
template <bool BF16>
__global__ __launch_bounds__(256) void saved_write_kernel(int64_t rows, int64_t cols, const void *x,
                                                          int64_t ldx, bool x_vec, uint8_t *codes,
                                                          int64_t ld, uint8_t *scales, int64_t lds,
                                                          bool s_vec, int64_t waves, int64_t col_waves)
{
    constexpr int NW = BF16 ? 4 : 8;
    const int64_t wv = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (wv >= waves)
        return;
    const Spot s = spot(wv, col_waves);
    const int n = (int)(cols - s.col < 8 ? cols - s.col : 8);
    const bool whole = x_vec && n == 8 && s.row + 8 <= rows;
    Raw<BF16> r[8];
    if (whole) {
        const char *p = static_cast<const char *>(x) + (s.row * ldx + s.col) * (BF16 ? 2 : 4);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int h = 0; h < NW / 4; ++h) {
                const uint4 v = *reinterpret_cast<const uint4 *>(p + i * ldx * (BF16 ? 2 : 4) + 16 * h);
                r[i].w[4 * h] = v.x, r[i].w[4 * h + 1] = v.y, r[i].w[4 * h + 2] = v.z, r[i].w[4 * h + 3] = v.w;
            }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (n > 0 && s.row + i < rows)
                load8(x, BF16, (s.row + i) * ldx + s.col, x_vec && n == 8, n, f);
#pragma unroll
            for (int k = 0; k < NW; ++k)
                r[i].w[k] = BF16 ? __float_as_uint(f[2 * k]) >> 16 | __float_as_uint(f[2 * k + 1])
                                 : __float_as_uint(f[k]);
        }
    }
    uint32_t m[NW];  // largest magnitude bits, packed as the input is
#pragma unroll
    for (int k = 0; k < NW; ++k) {
        m[k] = 0;
        auto more = [&](uint32_t u) {
            if (BF16)
                m[k] = __builtin_bit_cast(uint32_t,
                                          __builtin_elementwise_max(__builtin_bit_cast(u16x2, m[k]),
                                                                    __builtin_bit_cast(u16x2, u)));
            else
                m[k] = m[k] > u ? m[k] : u;
        };
#pragma unroll
        for (int i = 0; i < 8; ++i)
            more(r[i].w[k] & (BF16 ? 0x7fff7fffu : 0x7fffffffu));
#pragma unroll
        for (int d = 16; d < 64; d *= 2)
            more((uint32_t)__shfl_xor((int)m[k], d, 64));
    }
    uint32_t mx[8];
    bool special = false;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        mx[k] = BF16 ? (k & 1 ? m[(k >> 1) % NW] & 0xffff0000u : m[(k >> 1) % NW] << 16) : m[k % NW];
        special = special || mx[k] >= 0x7f700000u;
    }
    special = __any(special);
    if (special) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            mx[k] = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t u = mag_bits(r[i].at(k));
                mx[k] = u > mx[k] ? u : mx[k];
            }
#pragma unroll
            for (int d = 16; d < 64; d *= 2) {
                const uint32_t u = (uint32_t)__shfl_xor((int)mx[k], d, 64);
                mx[k] = u > mx[k] ? u : mx[k];
            }
        }
    }
    if (n <= 0)
        return;
    uint32_t byte[8];
    float inv[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        byte[k] = block_byte(mx[k]);
        inv[k] = inv_scale(byte[k]);
    }
    if (s.rg == 0)
        store_bytes8(scales + s.block * lds + s.col, s_vec && n == 8, n,
                     make_uint2(byte[0] | byte[1] << 8 | byte[2] << 16 | byte[3] << 24,
                                byte[4] | byte[5] << 8 | byte[6] << 16 | byte[7] << 24));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (!whole && s.row + i >= rows)
            break;
        float q[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            q[k] = (special ? coder_in(r[i].at(k)) : r[i].at(k)) * inv[k];
        store_bytes8(codes + (s.row + i) * ld + s.col, n == 8, n,
                     make_uint2(code4(q[0], q[1], q[2], q[3]), code4(q[4], q[5], q[6], q[7])));
    }
}

__global__ __launch_bounds__(256) void saved_read_kernel(int64_t rows, int64_t cols, const uint8_t *codes,
                                                         int64_t ld, const uint8_t *scales, int64_t lds,
                                                         bool s_vec, void *out, int64_t ldo, bool o_bf16,
                                                         bool o_vec, int64_t waves, int64_t col_waves)
{
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (w >= waves)
        return;
    const Spot s = spot(w, col_waves);
    const int n = (int)(cols - s.col < 8 ? cols - s.col : 8);
    if (n <= 0)
        return;
    const uint2 b = load_bytes8(scales + s.block * lds + s.col, s_vec && n == 8, n);
    uint2 c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        c[i] = s.row + i < rows ? load_bytes8(codes + (s.row + i) * ld + s.col, n == 8, n) : make_uint2(0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (s.row + i >= rows)
            break;
        float v[8];
        decode8(c[i], b, v);
        store8(out, o_bf16, (s.row + i) * ldo + s.col, o_vec && n == 8, n, v);
    }
}

struct ActBackArgs {
    int64_t rows, cols, ldy, ldz, ldd, ldzs;
    const void *dy;
    const void *z;
    const uint8_t *z_scales;
    void *dz;
    float *sums;  // dbias when one block spans the rows, else one row of partial sums per block
    int32_t units;  // of 128 rows, a block's walk
    bool y_bf16, y_vec, z_vec, zs_vec, d_vec;
    bool plain;  // bf16 dy, and every matrix's rows 16-byte aligned
};

// dz = dy act'(z) and the column sums of dz.  A block covers 128 columns of
// `units` x 128 rows: thread = 8 columns of 8 rows a unit (rows of one
// 32-row block, so one exponent load serves them), every access 16 bytes, or
// 8 for codes.  The sums stay in registers over the units, then go through
// LDS in row order and leave as one row per block, summed by sum_kernel in
// row order too: no atomics, the same bits every time.
//
// 4096 x 14336 with gelu and z in bf16: 71 us, 5.0 TB/s -- a plain copy on the
// same part runs at 4.8 to 5.0 -- and 5 us for the sums of the 32 blocks.
// With z in 8 bits 61 us (4.8 TB/s); with dy in fp32, which goes by rows without
// the loads ahead, 93 (5.0 TB/s).
// Besides memory the vector unit bounds it: gelu's slope is some 30 issue slots
// an element (its exponential and reciprocal go at a quarter of the rate), 42 us
// of the 71.
// ZF 0: no activation, 1: z in bf16, 2: z in 8 bits.
template <int ZF, int ACT>
__global__ __launch_bounds__(256) void act_backward_kernel(ActBackArgs p)
{
    __shared__ float part[16][128 + 4];
    const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
    const int64_t col = (int64_t)blockIdx.x * 128 + cg * 8;
    const int n = (int)(p.cols - col < 8 ? p.cols - col : 8);
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (n > 0) {
        for (int u = 0; u < p.units; ++u) {
            const int64_t row = ((int64_t)blockIdx.y * p.units + u) * 128 + rg * 8;
            if (row >= p.rows)
                break;
            uint2 b = make_uint2(0, 0);
            if (ZF == 2)
                b = load_bytes8(p.z_scales + (row >> 5) * p.ldzs + col, p.zs_vec && n == 8, n);
            auto finish = [&](int i, float (&y)[8], const float (&z)[8], bool vec) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if (ZF != 0)
                        y[k] *= act_slope<ACT>(z[k]);
                    sum[k] += y[k];
                }
                if (p.dz)
                    store8(p.dz, true, (row + i) * p.ldd + col, vec, n, y);
            };
            if (p.plain && n == 8 && row + 8 <= p.rows) {
                // every load of the unit before the first use
                uint4 wy[8], wz[ZF == 1 ? 8 : 1];
                uint2 wc[ZF == 2 ? 8 : 1];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    wy[i] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.dy) +
                                                             (row + i) * p.ldy + col);
                    if (ZF == 1)
                        wz[ZF == 1 ? i : 0] = *reinterpret_cast<const uint4 *>(
                            static_cast<const uint16_t *>(p.z) + (row + i) * p.ldz + col);
                    if (ZF == 2)
                        wc[ZF == 2 ? i : 0] = *reinterpret_cast<const uint2 *>(
                            static_cast<const uint8_t *>(p.z) + (row + i) * p.ldz + col);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float y[8], z[8] = {};
                    widen8(wy[i], y);
                    if (ZF == 1)
                        widen8(wz[ZF == 1 ? i : 0], z);
                    if (ZF == 2)
                        decode8(wc[ZF == 2 ? i : 0], b, z);
                    finish(i, y, z, true);
                }
                continue;
            }
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
                if (row + i >= p.rows)
                    break;
                float y[8], z[8] = {};
                load8(p.dy, p.y_bf16, (row + i) * p.ldy + col, p.y_vec && n == 8, n, y);
                if (ZF == 1)
                    load8(p.z, true, (row + i) * p.ldz + col, p.z_vec && n == 8, n, z);
                if (ZF == 2)
                    decode8(load_bytes8(static_cast<const uint8_t *>(p.z) + (row + i) * p.ldz + col, n == 8,
                                        n),
                            b, z);
                finish(i, y, z, p.d_vec && n == 8);
            }
        }
    }
    if (!p.sums)
        return;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        part[rg][cg * 8 + k] = sum[k];
    __syncthreads();
    const int64_t c = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (threadIdx.x < 128 && c < p.cols) {
        float s = 0.0f;
#pragma unroll
        for (int r = 0; r < 16; ++r)
            s += part[r][threadIdx.x];
        p.sums[(int64_t)blockIdx.y * p.cols + c] = s;
    }
}

// out[c] = sum of n rows of partial sums: 64 columns a block, its four waves a
// quarter of the rows each, the quarters added in order.
__global__ __launch_bounds__(256) void sum_kernel(const float *__restrict__ part, int64_t n, int64_t cols,
                                                  float *__restrict__ out)
{
    __shared__ float quarter[4][64];
    const int lane = threadIdx.x & 63, q = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    const int64_t per = (n + 3) / 4, end = (q + 1) * per < n ? (q + 1) * per : n;
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int64_t r = q * per; r < end; ++r)
            s += part[r * cols + c];
    }
    quarter[q][lane] = s;
    __syncthreads();
    if (q == 0 && c < cols)
        out[c] = ((quarter[0][lane] + quarter[1][lane]) + quarter[2][lane]) + quarter[3][lane];
}

}  // namespace

zero_status saved_check(const char *what, const zero_saved *s, int64_t rows, int64_t cols)
{
    if (!s)
        return fail(ZERO_ERR_INVALID_ARG, "%s is required", what);
    if (s->format != ZERO_SAVED_BF16 && s->format != ZERO_SAVED_E4M3)
        return fail(ZERO_ERR_INVALID_ARG, "%s: unknown format %d", what, s->format);
    zero_status st;
    if ((st = check_extent(rows, cols, s->ld)) != ZERO_OK)
        return st;
    if (rows == 0 && !s->data)
        return ZERO_OK;
    if (s->format == ZERO_SAVED_BF16)
        return check_matrix(what, s->data, s->ld, cols, ZERO_BF16);
    if (!s->data || !s->scales)
        return fail(ZERO_ERR_INVALID_ARG, "%s: codes and scales are required", what);
    if (s->ld < cols || s->ld_scales < cols)
        return fail(ZERO_ERR_INVALID_ARG, "%s: leading dimension below %lld columns", what, (long long)cols);
    if (s->ld % 16)
        return fail(ZERO_ERR_UNSUPPORTED, "%s: the codes' leading dimension must be a multiple of 16", what);
    if (s->ld_scales > kMaxDim)
        return fail(ZERO_ERR_UNSUPPORTED, "%s: the scales' leading dimension is too large", what);
    if (!aligned(s->data, 16))
        return fail(ZERO_ERR_ALIGNMENT, "%s: codes must be 16-byte aligned", what);
    return ZERO_OK;
}

// Rows a block of act_backward_kernel sums: enough that at most 64 rows of
// partial sums are left.
static int64_t act_units(int64_t rows)
{
    const int64_t u = (rows + 127) / 128;
    return u <= 64 ? 1 : (u + 63) / 64;
}

static int64_t act_blocks(int64_t rows)
{
    const int64_t per = 128 * act_units(rows);
    return (rows + per - 1) / per;
}

zero_status act_backward_check(int64_t rows, int64_t cols, const void *dy, int64_t ldy, int32_t dy_dtype,
                               int32_t act, const zero_saved *preact, const uint16_t *dz, int64_t ldz,
                               const float *dbias, const float *workspace, int64_t n_workspace)
{
    zero_status st;
    if ((st = check_extent(rows, cols, ldy)) != ZERO_OK || (st = check_extent(rows, cols, ldz)) != ZERO_OK)
        return st;
    if (act < ZERO_ACT_NONE || act > ZERO_ACT_SILU)
        return fail(ZERO_ERR_INVALID_ARG, "unknown activation %d", act);
    if (!known_dtype(dy_dtype))
        return fail(ZERO_ERR_INVALID_ARG, "dy: unknown dtype %d", dy_dtype);
    if (cols == 0)
        return ZERO_OK;
    if (rows > 0) {
        if ((st = check_matrix("dy", dy, ldy, cols, dy_dtype)) != ZERO_OK)
            return st;
        if (act != ZERO_ACT_NONE && (st = saved_check("preact", preact, rows, cols)) != ZERO_OK)
            return st;
        if (!dz && (act != ZERO_ACT_NONE || !dbias))
            return fail(ZERO_ERR_INVALID_ARG, "dz is required");
        if (dz && (st = check_matrix("dz", dz, ldz, cols, ZERO_BF16)) != ZERO_OK)
            return st;
        // In place of dy or of a bf16 z each element is read before it is
        // written; with another type or row length it would not be.
        if (dz && dz == dy && (dy_dtype != ZERO_BF16 || ldz != ldy))
            return fail(ZERO_ERR_INVALID_ARG, "dz in place of dy needs bf16 and the same leading dimension");
        if (dz && act != ZERO_ACT_NONE && dz == preact->data &&
            (preact->format != ZERO_SAVED_BF16 || ldz != preact->ld))
            return fail(ZERO_ERR_INVALID_ARG, "dz in place of preact needs bf16 and the same leading dimension");
    }
    if (!aligned(dbias, 4) || !aligned(workspace, 4))
        return fail(ZERO_ERR_ALIGNMENT, "dbias and workspace must be 4-byte aligned");
    const int64_t need = dbias ? zero_act_backward_workspace(rows, cols) : 0;
    if (need > 0 && (!workspace || n_workspace < need))
        return fail(ZERO_ERR_INVALID_ARG, "dbias of %lld x %lld needs a workspace of %lld floats",
                    (long long)rows, (long long)cols, (long long)need);
    if (rows > 0) {
        const bool kept = act != ZERO_ACT_NONE;
        const void *z = kept ? data_of(preact) : nullptr, *z_scales = kept ? scales_of(preact) : nullptr;
        const void *w = need > 0 ? workspace : nullptr;
        if (is_one_of(dbias, {dy, z, z_scales, dz, w}) || is_one_of(w, {dy, z, z_scales, dz}) ||
            is_one_of(dz, {z_scales}))
            return fail(ZERO_ERR_INVALID_ARG, "dz, dbias and the workspace need memory apart from what the "
                        "call reads and from each other");
    }
    if ((cols + 127) / 128 > int64_t(0x7fffffff) / 256)
        return fail(ZERO_ERR_UNSUPPORTED, "too many columns for one launch");
    return ZERO_OK;
}

zero_status act_backward_run(int64_t rows, int64_t cols, const void *dy, int64_t ldy, int32_t dy_dtype,
                             int32_t act, const zero_saved *preact, uint16_t *dz, int64_t ldz, float *dbias,
                             float *workspace, hipStream_t s)
{
    if (cols == 0 || (rows == 0 && !dbias))
        return ZERO_OK;
    ActBackArgs p = {};
    p.rows = rows;
    p.cols = cols;
    p.dy = dy;
    p.ldy = ldy;
    p.y_bf16 = dy_dtype == ZERO_BF16;
    p.y_vec = vec16(dy, ldy, bytes_of(dy_dtype));
    p.dz = dz;
    p.ldd = ldz;
    p.d_vec = vec16(dz, ldz, 2);
    if (act != ZERO_ACT_NONE && rows > 0) {
        p.z = preact->data;
        p.ldz = preact->ld;
        p.z_vec = vec16(preact->data, preact->ld, 2);
        if (preact->format == ZERO_SAVED_E4M3) {
            p.z_scales = preact->scales;
            p.ldzs = preact->ld_scales;
            p.zs_vec = aligned(p.z_scales, 8) && p.ldzs % 8 == 0;
        }
    }
    p.plain = p.y_bf16 && p.y_vec && (!p.z || p.z_scales || p.z_vec) && (!dz || p.d_vec);
    const int64_t blocks = rows > 0 ? act_blocks(rows) : 1;
    p.units = (int32_t)act_units(rows);
    p.sums = !dbias ? nullptr : blocks > 1 ? workspace : dbias;
    const dim3 grid((unsigned)((cols + 127) / 128), (unsigned)blocks);
    (void)hipGetLastError();
    by_act(p.z ? act : ZERO_ACT_NONE, [&](auto a) {
        constexpr int ACT = decltype(a)::value;
        if (ACT == ZERO_ACT_NONE)
            hipLaunchKernelGGL((act_backward_kernel<0, ZERO_ACT_NONE>), grid, dim3(256), 0, s, p);
        else if (p.z_scales)
            hipLaunchKernelGGL((act_backward_kernel<2, ACT>), grid, dim3(256), 0, s, p);
        else
            hipLaunchKernelGGL((act_backward_kernel<1, ACT>), grid, dim3(256), 0, s, p);
    });
    zero_status st = launched("act_backward");
    if (st != ZERO_OK || !dbias || blocks == 1)
        return st;
    hipLaunchKernelGGL(sum_kernel, dim3((unsigned)((cols + 63) / 64)), dim3(256), 0, s, workspace, blocks, cols,
                       dbias);
    return launched("dbias");
}

}  // namespace zs

extern "C" {

zero_status zero_saved_write(int64_t rows, int64_t cols, const void *x, int64_t ldx, int32_t x_dtype,
                             const zero_saved *out, void *stream)
{
    using namespace zs;
    zero_status st;
    if ((st = check_extent(rows, cols, ldx)) != ZERO_OK)
        return st;
    if (rows == 0 || cols == 0)
        return ZERO_OK;
    if ((st = check_matrix("x", x, ldx, cols, x_dtype)) != ZERO_OK ||
        (st = saved_check("out", out, rows, cols)) != ZERO_OK)
        return st;
    if (out->format != ZERO_SAVED_E4M3)
        return fail(ZERO_ERR_UNSUPPORTED, "only the 8-bit format is written from a matrix");
    if (is_one_of(out->data, {x, out->scales}) || out->scales == x)
        return fail(ZERO_ERR_INVALID_ARG, "a checkpoint needs a buffer of its own");
    const int64_t cw = (cols + 127) / 128, rb = (rows + 31) / 32;
    if (rb > int64_t(0x7fffffff) / 64 / cw)
        return fail(ZERO_ERR_UNSUPPORTED, "matrix too large for one launch");
    (void)hipGetLastError();
    const dim3 grid((unsigned)((rb * cw + 3) / 4));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    uint8_t *codes = static_cast<uint8_t *>(out->data);
    const bool xv = vec16(x, ldx, bytes_of(x_dtype));
    const bool sv = aligned(out->scales, 8) && out->ld_scales % 8 == 0;
    if (x_dtype == ZERO_BF16)
        hipLaunchKernelGGL(saved_write_kernel<true>, grid, dim3(256), 0, s, rows, cols, x, ldx, xv, codes,
                           out->ld, out->scales, out->ld_scales, sv, rb * cw, cw);
    else
        hipLaunchKernelGGL(saved_write_kernel<false>, grid, dim3(256), 0, s, rows, cols, x, ldx, xv, codes,
                           out->ld, out->scales, out->ld_scales, sv, rb * cw, cw);
    return launched("saved_write");
}

zero_status zero_saved_read(int64_t rows, int64_t cols, const zero_saved *in, void *out, int64_t ldo,
                            int32_t out_dtype, void *stream)
{
    using namespace zs;
    zero_status st;
    if ((st = check_extent(rows, cols, ldo)) != ZERO_OK)
        return st;
    if (rows == 0 || cols == 0)
        return ZERO_OK;
    if ((st = check_matrix("out", out, ldo, cols, out_dtype)) != ZERO_OK ||
        (st = saved_check("in", in, rows, cols)) != ZERO_OK)
        return st;
    if (in->format != ZERO_SAVED_E4M3)
        return fail(ZERO_ERR_UNSUPPORTED, "only the 8-bit format is read back");
    if (is_one_of(out, {in->data, in->scales}))
        return fail(ZERO_ERR_INVALID_ARG, "a checkpoint is not read back in place");
    const int64_t cw = (cols + 127) / 128, rb = (rows + 31) / 32;
    if (rb > int64_t(0x7fffffff) / 64 / cw)
        return fail(ZERO_ERR_UNSUPPORTED, "matrix too large for one launch");
    (void)hipGetLastError();
    hipLaunchKernelGGL(saved_read_kernel, dim3((unsigned)((rb * cw + 3) / 4)), dim3(256), 0,
                       static_cast<hipStream_t>(stream), rows, cols,
                       static_cast<const uint8_t *>(in->data), in->ld, in->scales, in->ld_scales,
                       aligned(in->scales, 8) && in->ld_scales % 8 == 0, out, ldo, out_dtype == ZERO_BF16,
                       vec16(out, ldo, bytes_of(out_dtype)), rb * cw, cw);
    return launched("saved_read");
}

int64_t zero_act_backward_workspace(int64_t rows, int64_t cols)
{
    if (rows <= 0 || cols <= 0)
        return 0;
    const int64_t b = zs::act_blocks(rows);
    return b > 1 ? b * cols : 0;
}

zero_status zero_act_backward(int64_t rows, int64_t cols, const void *dy, int64_t ldy, int32_t dy_dtype,
                              int32_t act, const zero_saved *preact, uint16_t *dz, int64_t ldz, float *dbias,
                              float *workspace, int64_t n_workspace, void *stream)
{
    const zero_status st = zs::act_backward_check(rows, cols, dy, ldy, dy_dtype, act, preact, dz, ldz, dbias,
                                                  workspace, n_workspace);
    if (st != ZERO_OK)
        return st;
    return zs::act_backward_run(rows, cols, dy, ldy, dy_dtype, act, preact, dz, ldz, dbias, workspace,
                                static_cast<hipStream_t>(stream));
}

}  // extern "C"
