// Softmax cross entropy of a linear head, z = x W over a large vocabulary, without
// the logits in memory.
//
//   lse_r  = log sum over c of exp z_rc,   loss_r = lse_r - z_r,target
//   dz_rc  = (exp(z_rc - lse_r) - [c = target_r]) dloss_r
//   dx     = dz W^T,   dW = x^T dz
// and loss_r = 0, dz_r = 0 for a target outside [0, vocab).
//
// Loss.  The product runs on the tiles of gemm_tile.h; its epilogue reduces each
// row of a tile to its maximum and the sum of exp(z - maximum), 8 bytes for 128 or
// 256 logits, and picks out the target's logit.  A second kernel joins a row's
// tiles.  All of it is fp32, from the accumulators on.
//
// Gradient.  The logits are computed again, a piece of the vocabulary at a time,
// the epilogue turning them into dz of the piece; dW of the piece and the piece's
// part of dx are products from it.  dz is rounded to bf16, as any linear layer's
// gradient is where a product reads it: half a step of 2^-8 of each dz, on terms
// that the sums of dx and dW add with independent errors.  The target's term, which
// outweighs the others, would carry the rounding of dloss, the same in every row of a
// mean; so dz is divided by the mantissa of a counting row's dloss, which leaves
// a common dloss a power of two, and dx and dW are multiplied by it in fp32 (100 rows
// over 50257 words, against 64-bit dx and dW: 3.2e-3 off without, 1.7e-3 with, which is
// what their own rounding to bf16 makes; results in fp32, 7e-5 off under a mean, 1.8e-3
// where each row has a dloss of its own, whose target's term rounds).  dx adds up over the pieces in fp32 and is
// rounded once.  Four products of 2 rows x vocab x hidden operations each, with the loss:
// 4096 tokens, 8192 x 128256, 26.2 ms, 1.31 PF/s, the rate of a plain product of this
// size; 100 tokens, 768 x 50257, 115 us, most of it one read of W for each product of
// few tiles.
//
// A vocabulary that is no multiple of 8 (stored with the vocabulary as rows) leaves
// up to 7 columns that the products' 16-byte reads cannot end at; their part of dx is a
// sum of its own.
#include <hip/hip_runtime.h>

#include <cmath>

#include "checks.h"
#include "gemm_place.h"
#include "products.h"
#include "vec.h"

namespace zs {
namespace {

constexpr float kLog2E = 1.4426950408889634f;
constexpr int kLoss = 0, kGrad = 1;

struct XentArgs {
    const int64_t *targets;
    int64_t vocab, c0;   // the first column of the piece
    float2 *part;        // loss: (maximum, sum) of each row of a tile column
    float *hit;          // loss: the targets' logits
    const float *lse, *dloss;
    uint16_t *dz;
    int64_t ldz;
};

// What the epilogue needs of the block's rows, fetched before the K loop.
struct RowLds {
    int target[kBM];   // the target's column within the piece, far off if none
    float lse[kBM], dloss[kBM];
    float mx[4][kBM], sum[4][kBM];  // loss: each column wave's part
};
constexpr int kNoTarget = -(1 << 30);

// The scale of dz: the mantissa, in [1, 2), of a counting row's dloss, the same row for
// every wave that asks: the first of 256 that lie evenly over the rows.  1 where none of
// them counts and has a normal number.  begin() reads, end() waits and decides.
struct ScaleOf {
    int64_t t[4], vocab;
    uint32_t u[4];

    __device__ __forceinline__ void begin(const int64_t *targets, const float *dloss, int64_t rows, int64_t words)
    {
        const int64_t step = rows < 512 ? 1 : rows / 256;
        vocab = words;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t row = (64 * k + (threadIdx.x & 63)) * step;
            t[k] = row < rows ? targets[row] : -1;
            u[k] = row < rows ? __float_as_uint(dloss[row]) & 0x7fffffffu : 0u;
        }
    }

    __device__ __forceinline__ float end() const
    {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint64_t good = __ballot(t[k] >= 0 && t[k] < vocab && u[k] >= 0x00800000u && u[k] < 0x7f800000u);
            if (good) {
                const uint32_t m = (uint32_t)__builtin_amdgcn_readlane((int)u[k], __builtin_ctzll(good));
                return __uint_as_float((m & 0x7fffffu) | 0x3f800000u);
            }
        }
        return 1.0f;
    }
};

template <int MODE>
__device__ __forceinline__ void fetch_rows(const XentArgs &p, int64_t m0, int64_t M, ZS_LDS RowLds *l)
{
    float scale = 1.0f;
    if constexpr (MODE == kGrad) {
        ScaleOf of;
        of.begin(p.targets, p.dloss, M, p.vocab);
        scale = of.end();
    }
    for (int i = threadIdx.x; i < kBM; i += kGT) {
        const int64_t row = m0 + i;
        const int64_t t = row < M ? p.targets[row] : -1;
        const bool valid = t >= 0 && t < p.vocab;
        const int64_t c = t - p.c0;
        // a valid target outside the piece still gives a gradient
        l->target[i] = !valid ? kNoTarget : c < -1 || c > 0x3fffffff ? -1 : (int)c;
        if (MODE == kGrad) {
            l->lse[i] = row < M ? p.lse[row] : 0.0f;
            l->dloss[i] = row < M ? p.dloss[row] / scale : 0.0f;
        }
    }
}

__device__ __forceinline__ float swap1(float x)  // of the neighbouring lane
{
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0xB1, 0xf, 0xf, true));
}

// Shift of a sum of exponentials about the maximum m: an empty one has m = -inf.
__device__ __forceinline__ float finite_max(float m) { return m == -__builtin_inff() ? 0.0f : m; }

template <int MODE>
struct XentEpi {
    const XentArgs &p;
    ZS_LDS float *lds;  // 32 * (CW + 4) floats of this wave
    ZS_LDS RowLds *rows;

    // 32 rows x CW columns in LDS, two lanes a row.  r0: the rows' first within the
    // block.
    template <int CW>
    __device__ __forceinline__ void loss_rows(int64_t row0, int r0, int64_t col0, int64_t M, int64_t N, int lane) const
    {
        constexpr int H = CW / 2;
        const int r = lane >> 1, h = lane & 1;
        const ZS_LDS float *q = lds + r * (CW + 4) + h * H;
        const int64_t left = N - col0 - h * H;
        const int n = left < 0 ? 0 : left < H ? (int)left : H;
        float x[H], m = -__builtin_inff(), s = 0.0f;
#pragma unroll
        for (int i = 0; i < H; i += 4) {
            const f32x4 v = *reinterpret_cast<const ZS_LDS f32x4 *>(q + i);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                x[i + k] = v[k];
        }
        if (n < H) {
#pragma unroll
            for (int i = 0; i < H; ++i)
                x[i] = i < n ? x[i] : -__builtin_inff();
        }
#pragma unroll
        for (int i = 0; i < H; ++i)
            m = __builtin_fmaxf(m, x[i]);
        m = __builtin_fmaxf(m, swap1(m));
        const float f = finite_max(m);
#pragma unroll
        for (int i = 0; i < H; ++i)
            s += __builtin_amdgcn_exp2f((x[i] - f) * kLog2E);
        s += swap1(s);
        const int64_t c = rows->target[r0 + r] - col0 - h * H;
        if (c >= 0 && c < n && row0 + r < M)
            p.hit[row0 + r] = q[c];
        if (h == 0) {
            rows->mx[(threadIdx.x >> 6) & 3][r0 + r] = m;
            rows->sum[(threadIdx.x >> 6) & 3][r0 + r] = s;
        }
    }

    // dz of 32 rows x CW columns in LDS, eight columns a lane.  dz's rows end at a
    // multiple of 8, so the columns past N in a lane's eight are written, as 0.
    template <int CW>
    __device__ __forceinline__ void grad_rows(int64_t row0, int r0, int64_t col0, int64_t M, int64_t N, int lane) const
    {
        constexpr int LPR = CW / 8, RPI = 64 / LPR, NP = 32 / RPI;
        const int64_t col = col0 + 8 * (lane % LPR);
        const int64_t left = N - col;
        if (left <= 0)
            return;
        const int n = left < 8 ? (int)left : 8;
#pragma unroll 1
        for (int it = 0; it < NP; ++it) {
            const int r = it * RPI + lane / LPR;
            if (row0 + r >= M)
                break;
            const ZS_LDS f32x4 *q = reinterpret_cast<const ZS_LDS f32x4 *>(lds + r * (CW + 4) + 8 * (lane % LPR));
            const f32x4 lo = q[0], hi = q[1];
            float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            const int t = rows->target[r0 + r];
            const float lse = rows->lse[r0 + r], d = rows->dloss[r0 + r];
            const int c = t - (int)col;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float e = __builtin_amdgcn_exp2f((x[k] - lse) * kLog2E);
                x[k] = t == kNoTarget || k >= n ? 0.0f : (c == k ? e - 1.0f : e) * d;
            }
            store8(p.dz, true, (row0 + r) * p.ldz + col, true, 8, x);
        }
    }

    template <int CW>
    __device__ __forceinline__ void rows32(int64_t row0, int r0, int64_t col0, int64_t M, int64_t N, int lane) const
    {
        wave_lds_order();
        if (MODE == kLoss)
            loss_rows<CW>(row0, r0, col0, M, N, lane);
        else
            grad_rows<CW>(row0, r0, col0, M, N, lane);
        wave_lds_order();
    }

    template <int I, int TM, int TN>
    __device__ __forceinline__ void step32(const f32x16 (&acc)[TM][TN], int64_t row0, int r0, int64_t col0, int64_t M,
                                           int64_t N, int lane) const
    {
        if constexpr (I < TM) {
            constexpr int CW = 32 * TN;
            const int fr = lane & 31, fh = lane >> 5;
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    lds[(8 * (v >> 2) + 4 * fh + (v & 3)) * (CW + 4) + 32 * j + fr] = acc[I][j][v];
            rows32<CW>(row0 + 32 * I, r0 + 32 * I, col0, M, N, lane);
            step32<I + 1>(acc, row0, r0, col0, M, N, lane);
        }
    }

    template <int I, int TM, int TN>
    __device__ __forceinline__ void step16(const f32x4 (&acc)[TM][TN], int64_t row0, int r0, int64_t col0, int64_t M,
                                           int64_t N, int lane) const
    {
        if constexpr (I < TM) {
            constexpr int CW = 16 * TN;
            const int r16 = lane & 15, g = lane >> 4;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        lds[(16 * h + 4 * g + v) * (CW + 4) + 16 * j + r16] = acc[I + h][j][v];
            rows32<CW>(row0 + 16 * I, r0 + 16 * I, col0, M, N, lane);
            step16<I + 2>(acc, row0, r0, col0, M, N, lane);
        }
    }

    // The four column waves' parts of BM rows, as one.
    template <int BM, int CW>
    __device__ __forceinline__ void join(int64_t m0, int64_t n0, int64_t M) const
    {
        if (MODE != kLoss)
            return;
        __syncthreads();
        const int t = threadIdx.x;
        if (t >= BM || m0 + t >= M)
            return;
        float m = -__builtin_inff(), s = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w)
            m = __builtin_fmaxf(m, rows->mx[w][t]);
        const float f = finite_max(m);
#pragma unroll
        for (int w = 0; w < 4; ++w)
            s += rows->sum[w][t] * __builtin_amdgcn_exp2f((rows->mx[w][t] - f) * kLog2E);
        p.part[n0 / (4 * CW) * M + m0 + t] = make_float2(m, s);
    }

    template <int TM, int TN>
    __device__ __forceinline__ void tile32(const f32x16 (&acc)[TM][TN], int64_t row0, int64_t col0, int64_t M,
                                           int64_t N, int lane) const
    {
        constexpr int CW = 32 * TN, HM = 32 * TM;
        const int wave = threadIdx.x >> 6, r0 = (wave >> 2) * HM;
        __syncthreads();  // every wave is done with the K loop's LDS
        step32<0>(acc, row0, r0, col0, M, N, lane);
        join<2 * HM, CW>(row0 - r0, col0 - (wave & 3) * CW, M);
    }

    template <int TM, int TN>
    __device__ __forceinline__ void tile16(const f32x4 (&acc)[TM][TN], int64_t row0, int64_t col0, int64_t M,
                                           int64_t N, int lane) const
    {
        constexpr int CW = 16 * TN, HM = 16 * TM;
        const int wave = threadIdx.x >> 6, r0 = (wave >> 2) * HM;
        __syncthreads();
        step16<0>(acc, row0, r0, col0, M, N, lane);
        join<2 * HM, CW>(row0 - r0, col0 - (wave & 3) * CW, M);
    }
};

// The vocabulary as rows of W: both operands K-inner.
template <int BM, int BN, int MODE>
__global__ __launch_bounds__(kGT) void xent_kernel_kp(int64_t M, int64_t N, int64_t K, const uint16_t *__restrict__ A,
                                                      int64_t lda, const uint16_t *__restrict__ B, int64_t ldb,
                                                      XentArgs args, int tiles_m, int tiles_n, int n_big)
{
    ZS_PAIRS(BM, BN);
    __shared__ RowLds rows;
    const XentEpi<MODE> epi{args, ZS_CORNER_KP(BN * 64), (ZS_LDS RowLds *)&rows};
    int64_t m0, n0;
    const bool whole = place<BM, BN>(tiles_m, tiles_n, n_big, m0, n0);
    if (m0 >= M)
        return;
    fetch_rows<MODE>(args, m0, M, (ZS_LDS RowLds *)&rows);
    if (whole)
        gemm_tile_kp<BM, BN>(M, N, K, A, lda, B, ldb, epi, m0, n0, ZS_P);
    else if constexpr (BM == kBM)
        gemm_tile_kp<BM / 2, BN>(M, N, K, A, lda, B, ldb, epi, m0, n0, ZS_P);
}

// The vocabulary as columns of W, 256 at a time.
template <int MODE>
__global__ __launch_bounds__(kGT) void xent_kernel_ap(int64_t M, int64_t N, int64_t K, const uint16_t *__restrict__ A,
                                                      int64_t lda, const uint16_t *__restrict__ B, int64_t ldb,
                                                      XentArgs args, int tiles_m, int tiles_n, int n_big)
{
    __shared__ __attribute__((aligned(1024))) char pa0[kPair], pa1[kPair];
    __shared__ __attribute__((aligned(1024))) char b0[kStage], b1[kStage], b2[kStage], b3[kStage];
    ZS_LDS char *const Bs[kStages] = {(ZS_LDS char *)b0, (ZS_LDS char *)b1, (ZS_LDS char *)b2, (ZS_LDS char *)b3};
    __shared__ RowLds rows;
    const XentEpi<MODE> epi{args,
                            corner((ZS_LDS char *)pa0, (ZS_LDS char *)pa0 + kPair / 2, (ZS_LDS char *)pa1,
                                   (ZS_LDS char *)pa1 + kPair / 2, (ZS_LDS char *)b0, (ZS_LDS char *)b1,
                                   (ZS_LDS char *)b2, (ZS_LDS char *)b3),
                            (ZS_LDS RowLds *)&rows};
    int64_t m0, n0;
    const bool whole = place<kBM, kBN>(tiles_m, tiles_n, n_big, m0, n0);
    if (m0 >= M)
        return;
    fetch_rows<MODE>(args, m0, M, (ZS_LDS RowLds *)&rows);
    if (whole)
        gemm_tile_ap<kBM>(M, N, K, A, lda, B, ldb, epi, m0, n0, (ZS_LDS char *)pa0, (ZS_LDS char *)pa1, Bs);
    else
        gemm_tile_ap<kBM / 2>(M, N, K, A, lda, B, ldb, epi, m0, n0, (ZS_LDS char *)pa0, (ZS_LDS char *)pa1, Bs);
}

// The same in 128 x 128 tiles.
template <int MODE>
__global__ __launch_bounds__(kGT) void xent_kernel_small(int64_t M, int64_t N, int64_t K,
                                                         const uint16_t *__restrict__ A, int64_t lda,
                                                         const uint16_t *__restrict__ B, int64_t ldb, XentArgs args,
                                                         int tiles_m, int tiles_n, int n_big)
{
    ZS_STAGES(128, 128);
    __shared__ RowLds rows;
    const XentEpi<MODE> epi{args, ZS_CORNER, (ZS_LDS RowLds *)&rows};
    int64_t m0, n0;
    place<128, 128>(tiles_m, tiles_n, n_big, m0, n0);
    fetch_rows<MODE>(args, m0, M, (ZS_LDS RowLds *)&rows);
    gemm_tile<128, 128, false, true>(M, N, K, A, lda, B, ldb, epi, m0, n0, As, Bs);
}

// A row's tiles joined: 16 rows a block, 64 runs of tiles side by side.
__global__ __launch_bounds__(1024) void xent_join_kernel(const float2 *__restrict__ part, const float *__restrict__ hit,
                                                         const int64_t *__restrict__ targets, int64_t M, int n_tiles,
                                                         int64_t vocab, float *__restrict__ loss,
                                                         float *__restrict__ lse)
{
    __shared__ float ms[64][16], ss[64][16];
    const int c = threadIdx.x & 15, run = threadIdx.x >> 4;
    const int64_t row = (int64_t)blockIdx.x * 16 + c;
    const int per = (n_tiles + 63) / 64, t1 = (run + 1) * per < n_tiles ? (run + 1) * per : n_tiles;
    float m = -__builtin_inff(), s = 0.0f;
    auto add = [&](float x, float y) {
        const float n = __builtin_fmaxf(m, x), f = finite_max(n);
        s = s * __builtin_amdgcn_exp2f((m - f) * kLog2E) + y * __builtin_amdgcn_exp2f((x - f) * kLog2E);
        m = n;
    };
    if (row < M) {
#pragma unroll 8
        for (int t = run * per; t < t1; ++t) {
            const float2 a = part[t * M + row];
            add(a.x, a.y);
        }
    }
    ms[run][c] = m;
    ss[run][c] = s;
    __syncthreads();
    // halves of the runs, always in the same order
    for (int d = 32; d > 0; d /= 2) {
        if (run < d) {
            add(ms[run + d][c], ss[run + d][c]);
            ms[run][c] = m;
            ss[run][c] = s;
        }
        __syncthreads();
    }
    if (run > 0 || row >= M)
        return;
    const float l = m + logf(s);
    const int64_t t = targets[row];
    lse[row] = l;
    loss[row] = t >= 0 && t < vocab ? l - hit[row] : 0.0f;
}

__device__ __forceinline__ float bf16_of(const uint16_t *p, int64_t i) { return __uint_as_float((uint32_t)p[i] << 16); }

// dx of few rows: its tiles would leave most CUs idle over a sum as long as the
// vocabulary, so the sum is cut into runs of `per` words, a block each, whose fp32
// parts xent_dx_sum_kernel adds up in order.  128 x 128 tiles.
template <bool B_KOUTER>
__global__ __launch_bounds__(kGT) void xent_dx_kernel(int64_t M, int64_t N, int64_t K, int64_t per,
                                                      const uint16_t *__restrict__ dz, int64_t ldz,
                                                      const uint16_t *__restrict__ w, int64_t ldw, float *part,
                                                      int tiles_m, int tiles_n)
{
    // the tiles of a run, which share its dz, on one XCD
    const int b = xcd_order(blockIdx.x, gridDim.x), tiles = tiles_m * tiles_n, tile = b % tiles;
    const int64_t run = b / tiles, k0 = run * per;
    const int64_t k = K - k0 < per ? K - k0 : per;
    const PlainEpi<false> epi{part + run * M * N, N};
    const int64_t m0 = (int64_t)(tile % tiles_m) * 128, n0 = (int64_t)(tile / tiles_m) * 128;
    if constexpr (B_KOUTER) {
        ZS_STAGES(128, 128);
        gemm_tile<128, 128, false, true>(M, N, k, dz + k0, ldz, w + k0 * ldw, ldw, epi, m0, n0, As, Bs);
    } else {
        ZS_PAIRS(128, 128);
        gemm_tile_kp<128, 128>(M, N, k, dz + k0, ldz, w + k0, ldw, epi, m0, n0, ZS_P);
    }
}

// dx = acc + the runs' parts + the last n < 8 words' dz[r][c] W[c][h], times the scale of
// dz where `targets` are given.
struct DxOut {
    const uint16_t *dz, *w;
    int64_t ldz, ldw;
    const float *acc;
    int64_t ldacc;
    void *out;
    int64_t ldout;
    const int64_t *targets;
    const float *dloss;
    int64_t vocab;
    int n;
    bool bf16;

    __device__ __forceinline__ float scale(int64_t rows) const
    {
        if (!targets)
            return 1.0f;
        ScaleOf of;
        of.begin(targets, dloss, rows, vocab);
        return of.end();
    }

    __device__ __forceinline__ void store(int64_t r, int64_t h, float (&s)[8], float scale) const
    {
        float x[8];
        if (acc) {
            load8(acc, false, r * ldacc + h, true, 8, x);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s[e] += x[e];
        }
        for (int c = 0; c < n; ++c) {
            const float d = bf16_of(dz, r * ldz + c);
            load8(w, true, c * ldw + h, true, 8, x);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s[e] = __builtin_fmaf(d, x[e], s[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            s[e] *= scale;
        store8(out, bf16, r * ldout + h, true, 8, s);
    }
};

// 32 groups of eight values a block, its eight threads a group an eighth of the runs
// each, added in order.
__global__ __launch_bounds__(256) void xent_dx_sum_kernel(int64_t rows, int64_t hidden, int runs,
                                                          const float *__restrict__ part, DxOut p)
{
    __shared__ float eighth[8][8][32];
    const float scale = p.scale(rows);
    const int g = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int64_t per = hidden / 8, all = rows * per;
    const int each = (runs + 7) / 8, end = (q + 1) * each < runs ? (q + 1) * each : runs;
    for (int64_t i0 = (int64_t)blockIdx.x * 32; i0 < all; i0 += (int64_t)gridDim.x * 32) {
        const int64_t i = i0 + g, r = i / per, h = i % per * 8;
        float s[8] = {}, x[8];
        if (i < all) {
#pragma unroll 8
            for (int k = q * each; k < end; ++k) {
                load8(part, false, (k * rows + r) * hidden + h, true, 8, x);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    s[e] += x[e];
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            eighth[q][e][g] = s[e];
        __syncthreads();
        if (q == 0 && i < all) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
                for (int k = 1; k < 8; ++k)
                    s[e] += eighth[k][e][g];
            p.store(r, h, s, scale);
        }
        __syncthreads();
    }
}

// The same of one product, which is in acc: eight values a thread, 4096 x 8192 in 39 us,
// 5.2 TB/s (the kernel above, which has one thread in eight for this, 193).
__global__ __launch_bounds__(256) void xent_dx_out_kernel(int64_t rows, int64_t hidden, DxOut p)
{
    const float scale = p.scale(rows);
    const int64_t per = hidden / 8, all = rows * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        float s[8] = {};
        p.store(i / per, i % per * 8, s, scale);
    }
}

// dW = A^T B over K rows, times the scale of dz, stored in whole rows of 16 bytes a lane.
// M and N are rounded up to 8, which A and B hold; `m` and `n` are what is stored.
template <bool BF16>
struct StoreEpi {
    ZS_LDS float *lds;
    void *C;
    int64_t ldc, m, n;
    ScaleOf of;

    template <int I, int TM, int TN>
    __device__ __forceinline__ void step(const f32x16 (&acc)[TM][TN], int64_t row0, int64_t col0, int lane,
                                         float scale) const
    {
        if constexpr (I < TM) {
            constexpr int CW = 32 * TN, LPR = CW / 8, RPI = 64 / LPR;
            const int fr = lane & 31, fh = lane >> 5;
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    lds[(8 * (v >> 2) + 4 * fh + (v & 3)) * (CW + 4) + 32 * j + fr] = acc[I][j][v] * scale;
            wave_lds_order();
            const int64_t col = col0 + 8 * (lane % LPR), left = n - col;
            const int k = left <= 0 ? 0 : left < 8 ? (int)left : 8;
#pragma unroll
            for (int it = 0; it < 32 / RPI; ++it) {
                const int r = it * RPI + lane / LPR;
                if (row0 + 32 * I + r >= m || k == 0)
                    continue;
                const ZS_LDS f32x4 *q = reinterpret_cast<const ZS_LDS f32x4 *>(lds + r * (CW + 4) + 8 * (lane % LPR));
                const f32x4 lo = q[0], hi = q[1];
                const float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                store8(C, BF16, (row0 + 32 * I + r) * ldc + col, k == 8, k, x);
            }
            wave_lds_order();
            step<I + 1>(acc, row0, col0, lane, scale);
        }
    }

    template <int TM, int TN>
    __device__ __forceinline__ void tile32(const f32x16 (&acc)[TM][TN], int64_t row0, int64_t col0, int64_t, int64_t,
                                           int lane) const
    {
        __syncthreads();
        step<0>(acc, row0, col0, lane, of.end());
    }
};

struct DwArgs {
    void *C;
    int64_t ldc, m, n;
    const int64_t *targets;
    const float *dloss;
    int64_t vocab;
};

// BM: 256 (and halves), or 128 for few rows: short sums, so the stores are the work, and
// with two blocks a CU one's loads run under the other's stores.
template <int BM, bool BF16>
__global__ __launch_bounds__(kGT) void xent_dw_kernel(int64_t M, int64_t N, int64_t K, const uint16_t *__restrict__ A,
                                                      int64_t lda, const uint16_t *__restrict__ B, int64_t ldb,
                                                      DwArgs p, int tiles_m, int tiles_n, int n_big)
{
    ZS_STAGES(BM, BM);
    StoreEpi<BF16> epi{ZS_CORNER, p.C, p.ldc, p.m, p.n, {}};
    epi.of.begin(p.targets, p.dloss, K, p.vocab);
    int64_t m0, n0;
    if (place<BM, BM>(tiles_m, tiles_n, n_big, m0, n0))
        gemm_tile<BM, BM, true, true>(M, N, K, A, lda, B, ldb, epi, m0, n0, As, Bs);
    else if constexpr (BM == kBM)
        gemm_tile<BM / 2, BM, true, true>(M, N, K, A, lda, B, ldb, epi, m0, n0, As, Bs);
}

// Columns of a tile: 128 (of 128 rows, two blocks a CU) where 256 x 256 tiles would
// not fill half the CUs, or would be half empty.
int xent_bn(int64_t rows, int64_t cols) { return rows <= 128 || small_tiles(rows, cols) ? 128 : kBN; }

template <int MODE>
zero_status launch_xent(int64_t M, int64_t N, int64_t K, const uint16_t *x, int64_t ldx, const uint16_t *w, int64_t ldw,
                        bool outer, const XentArgs &a, hipStream_t s)
{
    (void)hipGetLastError();
#define ZS_XENT(KERNEL, G)                                                                         \
    hipLaunchKernelGGL(KERNEL, G.grid, dim3(kGT), 0, s, M, N, K, x, ldx, w, ldw, a, G.tm, G.tn, G.n_big)
    if (xent_bn(M, N) == 128) {
        const Grid g = tiles(M, N, 128, 128, false);
        if (outer)
            ZS_XENT((xent_kernel_small<MODE>), g);
        else
            ZS_XENT((xent_kernel_kp<128, 128, MODE>), g);
    } else {
        const Grid g = tiles(M, N, kBM, kBN, true);
        if (outer)
            ZS_XENT((xent_kernel_ap<MODE>), g);
        else
            ZS_XENT((xent_kernel_kp<kBM, kBN, MODE>), g);
    }
#undef ZS_XENT
    return launched("linear_xent");
}

// Columns of a piece: all pieces of one width but the last, which is narrower, at
// most `piece` wide.
int64_t piece_width(int64_t rows, int64_t vocab, int64_t piece)
{
    if (piece == 0) {
        // 128 MB of dz, and no pieces so narrow that adding dx up would show
        piece = rows > 0 ? ZERO_XENT_PIECE_ELEMS / rows / 256 * 256 : vocab;
        piece = piece < 4096 ? 4096 : piece;
    }
    if (piece >= vocab)
        return vocab;
    const int64_t n = (vocab + piece - 1) / piece;
    const int64_t even = ((vocab + n - 1) / n + 255) / 256 * 256;
    return even < piece ? even : piece;
}

// Runs that dx's sum over n words is cut into: two blocks a CU, at least 512 words
// each, where its tiles alone would not fill half the CUs; 1: no cut.  `room`: floats
// for their parts.
int64_t dx_runs(int64_t rows, int64_t hidden, int64_t n, int64_t room)
{
    const int64_t t = ((rows + 127) / 128) * ((hidden + 127) / 128), cus = cu_count();
    if (2 * t > cus)
        return 1;
    int64_t runs = 2 * cus / t;
    runs = runs < n / 512 ? runs : n / 512;
    runs = runs < room / (rows * hidden) ? runs : room / (rows * hidden);
    return runs < 2 ? 1 : runs;
}

int64_t forward_floats(int64_t rows, int64_t vocab)
{
    const int bn = xent_bn(rows, vocab);
    return rows * (2 * ((vocab + bn - 1) / bn) + 1);
}

int64_t backward_floats(int64_t rows, int64_t vocab, int64_t hidden, int64_t piece)
{
    const int64_t ldz = (piece_width(rows, vocab, piece) + 7) / 8 * 8;
    return rows * (ldz / 2) + rows * hidden;
}

// dW = A^T B (m x n over `rows` rows), A's rows holding up to 7 columns more.
zero_status run_dw(int64_t m, int64_t n, int64_t rows, const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb,
                   void *C, int64_t ldc, int32_t c_dtype, const int64_t *targets, const float *dloss, int64_t vocab,
                   hipStream_t s)
{
    const int64_t M = (m + 7) / 8 * 8;
    const DwArgs p = {C, ldc, m, n, targets, dloss, vocab};
    (void)hipGetLastError();
#define ZS_DW(BM, BF)                                                                              \
    hipLaunchKernelGGL((xent_dw_kernel<BM, BF>), g.grid, dim3(kGT), 0, s, M, n, rows, A, lda, B, ldb, p, g.tm, g.tn, \
                       g.n_big)
    // 100 rows, 50257 x 768: 33 us in 128 x 128 tiles and 40 in 256 x 256 ones, 33 rows, 4096
    // x 128256, 385 and 398; 256 rows 48 and 48, 666 and 615; 512 rows 66 and 62.
    if (rows <= 128 || small_tiles(M, n)) {
        const Grid g = tiles(M, n, 128, 128, false);
        if (c_dtype == ZERO_BF16)
            ZS_DW(128, true);
        else
            ZS_DW(128, false);
    } else {
        const Grid g = tiles(M, n, kBM, kBN, true);
        if (c_dtype == ZERO_BF16)
            ZS_DW(kBM, true);
        else
            ZS_DW(kBM, false);
    }
#undef ZS_DW
    return launched("linear_xent dw");
}

zero_status sum_dx(int64_t rows, int64_t hidden, int runs, const float *part, int tail, const uint16_t *dz, int64_t ldz,
                   const uint16_t *w, int64_t ldw, const float *acc, int64_t ldacc, void *out, int64_t ldout,
                   int32_t out_dtype, const int64_t *targets, const float *dloss, int64_t vocab, hipStream_t s)
{
    const DxOut p = {dz, w, ldz, ldw, acc, ldacc, out, ldout, targets, dloss, vocab, tail, out_dtype == ZERO_BF16};
    const int64_t eights = rows * (hidden / 8), each = runs > 0 ? 32 : 256;
    int64_t grid = (eights + each - 1) / each;
    // a block's scale, 1 us, before several rounds of it where there is no sum to wait for
    const int64_t most = runs > 0 ? 65536 : 2048;
    grid = grid > most ? most : grid;
    (void)hipGetLastError();
    if (runs > 0)
        hipLaunchKernelGGL(xent_dx_sum_kernel, dim3((unsigned)grid), dim3(256), 0, s, rows, hidden, runs, part, p);
    else
        hipLaunchKernelGGL(xent_dx_out_kernel, dim3((unsigned)grid), dim3(256), 0, s, rows, hidden, p);
    return launched("linear_xent dx sum");
}

zero_status check_piece(int64_t piece)
{
    if (piece < 0 || (piece > 0 && piece % 256))
        return fail(ZERO_ERR_INVALID_ARG, "piece must be 0 or a multiple of 256 words");
    return ZERO_OK;
}

// xent_join_kernel takes 1024 threads for 16 rows, and the dispatch counts a launch's
// threads in 32 bits.
constexpr int64_t kMaxRows = int64_t(0xffffffffu) / 1024 * 16;

// Sizes for which the workspace's own can be computed.
zero_status check_sizes(int64_t rows, int64_t vocab, int64_t hidden)
{
    if (rows < 0 || vocab < 1 || hidden < 1)
        return fail(ZERO_ERR_INVALID_ARG, "rows >= 0, vocab >= 1 and hidden >= 1 are required");
    if (rows > kMaxRows || vocab > (int64_t(1) << 30) || hidden > (int64_t(1) << 30))
        return fail(ZERO_ERR_UNSUPPORTED, "at most %lld rows, a vocab and hidden of 2^30", (long long)kMaxRows);
    return ZERO_OK;
}

zero_status check_common(int64_t rows, int64_t vocab, int64_t hidden, const uint16_t *x, int64_t ldx,
                         const uint16_t *w, int64_t ldw, int32_t w_order, const int64_t *targets)
{
    zero_status st;
    if ((st = check_sizes(rows, vocab, hidden)) != ZERO_OK)
        return st;
    if (rows > 0 && !targets)
        return fail(ZERO_ERR_INVALID_ARG, "targets are required");
    if (!aligned(targets, 8))
        return fail(ZERO_ERR_ALIGNMENT, "targets must be 8-byte aligned");
    alignas(16) static const float none[4] = {};
    return gemm_check(rows, vocab, hidden, x, ldx, ZERO_K_INNER, w, ldw, w_order, none, vocab, ZERO_FP32);
}

}  // namespace

zero_status xent_forward_check(int64_t rows, int64_t vocab, int64_t hidden, const uint16_t *x, int64_t ldx,
                               const uint16_t *w, int64_t ldw, int32_t w_order, const int64_t *targets,
                               const float *loss, const float *lse, const float *workspace, int64_t n_workspace)
{
    zero_status st;
    if ((st = check_common(rows, vocab, hidden, x, ldx, w, ldw, w_order, targets)) != ZERO_OK || rows == 0)
        return st;
    if (!loss || !lse)
        return fail(ZERO_ERR_INVALID_ARG, "loss and lse are required");
    const int64_t need = forward_floats(rows, vocab);
    if (!workspace || n_workspace < need)
        return fail(ZERO_ERR_INVALID_ARG, "the loss of %lld rows over %lld words needs a workspace of %lld floats",
                    (long long)rows, (long long)vocab, (long long)need);
    if (!aligned(loss, 4) || !aligned(lse, 4) || !aligned(workspace, 8))
        return fail(ZERO_ERR_ALIGNMENT, "loss and lse must be 4-byte aligned, the workspace 8-byte");
    if (is_one_of(loss, {x, w, targets, lse, workspace}) || is_one_of(lse, {x, w, targets, workspace}) ||
        is_one_of(workspace, {x, w, targets}))
        return fail(ZERO_ERR_INVALID_ARG, "loss, lse and the workspace need memory apart from what the call reads "
                    "and from each other");
    return ZERO_OK;
}

zero_status xent_forward_run(int64_t rows, int64_t vocab, int64_t hidden, const uint16_t *x, int64_t ldx,
                             const uint16_t *w, int64_t ldw, int32_t w_order, const int64_t *targets, float *loss,
                             float *lse, float *workspace, hipStream_t s)
{
    if (rows == 0)
        return ZERO_OK;
    const int bn = xent_bn(rows, vocab);
    const int n_tiles = (int)((vocab + bn - 1) / bn);
    XentArgs a = {};
    a.targets = targets;
    a.vocab = vocab;
    a.part = reinterpret_cast<float2 *>(workspace);
    a.hit = workspace + 2 * rows * n_tiles;
    zero_status st = launch_xent<kLoss>(rows, vocab, hidden, x, ldx, w, ldw, w_order == ZERO_K_OUTER, a, s);
    if (st != ZERO_OK)
        return st;
    hipLaunchKernelGGL(xent_join_kernel, dim3((unsigned)((rows + 15) / 16)), dim3(1024), 0, s, a.part, a.hit, targets,
                       rows, n_tiles, vocab, loss, lse);
    return launched("linear_xent join");
}

zero_status xent_backward_check(int64_t rows, int64_t vocab, int64_t hidden, const uint16_t *x, int64_t ldx,
                                const uint16_t *w, int64_t ldw, int32_t w_order, const int64_t *targets,
                                const float *lse, const float *dloss, const void *dx, int64_t lddx, int32_t dx_dtype,
                                const void *dw, int64_t lddw, int32_t dw_dtype, int64_t piece, const float *workspace,
                                int64_t n_workspace)
{
    zero_status st;
    if ((st = check_piece(piece)) != ZERO_OK || (st = check_sizes(rows, vocab, hidden)) != ZERO_OK)
        return st;
    const int64_t dw_cols = w_order == ZERO_K_OUTER ? vocab : hidden;
    if (!known_dtype(dx_dtype))
        return fail(ZERO_ERR_INVALID_ARG, "dx: unknown dtype %d", dx_dtype);
    if ((st = check_matrix("dw", dw, lddw, dw_cols, dw_dtype)) != ZERO_OK)
        return st;
    if (hidden % 8 || (w_order == ZERO_K_OUTER && vocab % 8))
        return fail(ZERO_ERR_UNSUPPORTED, "hidden, and a vocabulary stored as columns, must be multiples of 8");
    if (lddw > kMaxDim || lddx > kMaxDim)
        return fail(ZERO_ERR_UNSUPPORTED, "leading dimension too large");
    constexpr int64_t kMaxTiles = int64_t(0xffffffffu) / (2 * kGT);
    const int64_t th = (hidden + kBM - 1) / kBM, tv = (vocab + kBN - 1) / kBN, tr = (rows + kBM - 1) / kBM;
    if (th > kMaxTiles / tv || (tr > 0 && th > kMaxTiles / tr))
        return fail(ZERO_ERR_UNSUPPORTED, "too many tiles for one launch");
    if ((st = check_common(rows, vocab, hidden, x, ldx, w, ldw, w_order, targets)) != ZERO_OK || rows == 0)
        return st;
    if ((st = check_matrix("dx", dx, lddx, hidden, dx_dtype)) != ZERO_OK)
        return st;
    if (!lse || !dloss)
        return fail(ZERO_ERR_INVALID_ARG, "lse and dloss are required");
    // x is an operand with the rows as K, dz one with the words as K or as rows
    const int64_t ldz = (piece_width(rows, vocab, piece) + 7) / 8 * 8;
    if (ldx > (int64_t(1) << 25) || ldz > (int64_t(1) << 22) || (w_order == ZERO_K_OUTER && ldw > (int64_t(1) << 22)))
        return fail(ZERO_ERR_UNSUPPORTED, "leading dimension or piece too large for 32-bit operand offsets");
    const int64_t need = backward_floats(rows, vocab, hidden, piece);
    if (!workspace || n_workspace < need)
        return fail(ZERO_ERR_INVALID_ARG, "the gradient of %lld rows over %lld words needs a workspace of %lld floats",
                    (long long)rows, (long long)vocab, (long long)need);
    if (!aligned(lse, 4) || !aligned(dloss, 4) || !aligned(workspace, 16))
        return fail(ZERO_ERR_ALIGNMENT, "lse and dloss must be 4-byte aligned, the workspace 16-byte");
    if (is_one_of(dx, {x, w, targets, lse, dloss, dw, workspace}) ||
        is_one_of(dw, {x, w, targets, lse, dloss, workspace}) || is_one_of(workspace, {x, w, targets, lse, dloss}))
        return fail(ZERO_ERR_INVALID_ARG, "dx, dw and the workspace need memory apart from what the call reads and "
                    "from each other");
    return ZERO_OK;
}

zero_status xent_backward_run(int64_t rows, int64_t vocab, int64_t hidden, const uint16_t *x, int64_t ldx,
                              const uint16_t *w, int64_t ldw, int32_t w_order, const int64_t *targets,
                              const float *lse, const float *dloss, void *dx, int64_t lddx, int32_t dx_dtype, void *dw,
                              int64_t lddw, int32_t dw_dtype, int64_t piece, float *workspace, hipStream_t s)
{
    const bool outer = w_order == ZERO_K_OUTER;
    const int64_t width = piece_width(rows, vocab, piece), ldz = (width + 7) / 8 * 8;
    uint16_t *const dz = reinterpret_cast<uint16_t *>(workspace);
    // where dx adds up: itself, if it is fp32
    const bool own = dx_dtype == ZERO_FP32;
    float *const acc = own ? static_cast<float *>(dx) : workspace + rows * (ldz / 2);
    const int64_t ldacc = own ? lddx : hidden;
    const int es = bytes_of(dw_dtype);
    bool added = false;
    for (int64_t c0 = 0; c0 < vocab; c0 += width) {
        const int64_t n = vocab - c0 < width ? vocab - c0 : width, n8 = n / 8 * 8;
        const int tail = (int)(n - n8);
        const bool last = c0 + width >= vocab;
        const uint16_t *wp = w + (outer ? c0 : c0 * ldw);
        char *const dwp = static_cast<char *>(dw) + (outer ? c0 : c0 * lddw) * es;
        zero_status st;
        if (rows > 0) {
            XentArgs a = {};
            a.targets = targets, a.vocab = vocab, a.c0 = c0;
            a.lse = lse, a.dloss = dloss, a.dz = dz, a.ldz = ldz;
            if ((st = launch_xent<kGrad>(rows, n, hidden, x, ldx, wp, ldw, outer, a, s)) != ZERO_OK)
                return st;
        }
        const int32_t w_as_b = outer ? ZERO_K_INNER : ZERO_K_OUTER;
        if (rows > 0) {
            // dx's part goes first: until dW is there, its memory has room for runs
            const int64_t dw_cols = outer ? vocab : hidden;
            const bool free = lddw == dw_cols && (!outer || n == vocab) && aligned(dwp, 16);
            const int64_t runs = dx_runs(rows, hidden, n8, free ? n * hidden * es / 4 : 0);
            // the last piece leaves dx, scaled and in its type
            void *const to = last ? dx : acc;
            const int64_t ldto = last ? lddx : ldacc;
            const int32_t tt = last ? dx_dtype : ZERO_FP32;
            const int64_t *const scaled = last ? targets : nullptr;
            const uint16_t *const zt = dz + n8, *const wt = wp + n8 * ldw;
            if (runs > 1) {
                float *const part = reinterpret_cast<float *>(dwp);
                const int64_t per = ((n8 + runs - 1) / runs + 63) / 64 * 64, real = (n8 + per - 1) / per;
                const int tm = (int)((rows + 127) / 128), tn = (int)((hidden + 127) / 128);
                const dim3 grid((unsigned)(tm * tn * real));
                (void)hipGetLastError();
                if (outer)
                    hipLaunchKernelGGL((xent_dx_kernel<false>), grid, dim3(kGT), 0, s, rows, hidden, n8, per, dz, ldz, wp,
                                       ldw, part, tm, tn);
                else
                    hipLaunchKernelGGL((xent_dx_kernel<true>), grid, dim3(kGT), 0, s, rows, hidden, n8, per, dz, ldz, wp,
                                       ldw, part, tm, tn);
                if ((st = launched("linear_xent dx")) != ZERO_OK ||
                    (st = sum_dx(rows, hidden, (int)real, part, tail, zt, ldz, wt, ldw, added ? acc : nullptr, ldacc, to,
                                 ldto, tt, scaled, dloss, vocab, s)) != ZERO_OK)
                    return st;
            } else {
                zero_epilogue ep = {};
                ep.residual = acc;
                ep.ldr = ldacc;
                ep.residual_dtype = ZERO_FP32;
                if ((st = epilogue_gemm_run(rows, hidden, n8, dz, ldz, ZERO_K_INNER, wp, ldw, w_as_b, acc, ldacc,
                                            ZERO_FP32, added ? &ep : nullptr, s)) != ZERO_OK ||
                    ((last || tail > 0) &&
                     (st = sum_dx(rows, hidden, 0, nullptr, tail, zt, ldz, wt, ldw, acc, ldacc, to, ldto, tt, scaled,
                                  dloss, vocab, s)) != ZERO_OK))
                    return st;
            }
            added = true;
        }
        st = outer ? run_dw(hidden, n, rows, x, ldx, dz, ldz, dwp, lddw, dw_dtype, targets, dloss, vocab, s)
                   : run_dw(n, hidden, rows, dz, ldz, x, ldx, dwp, lddw, dw_dtype, targets, dloss, vocab, s);
        if (st != ZERO_OK)
            return st;
    }
    return ZERO_OK;
}

}  // namespace zs

extern "C" {

int64_t zero_linear_xent_workspace(int64_t rows, int64_t vocab, int64_t hidden, int32_t backward, int64_t piece)
{
    using namespace zs;
    if (check_sizes(rows, vocab, hidden) != ZERO_OK || check_piece(piece) != ZERO_OK || rows == 0)
        return 0;
    return backward ? backward_floats(rows, vocab, hidden, piece) : forward_floats(rows, vocab);
}

zero_status zero_linear_xent_forward(int64_t rows, int64_t vocab, int64_t hidden, const uint16_t *x, int64_t ldx,
                                     const uint16_t *w, int64_t ldw, int32_t w_order, const int64_t *targets,
                                     float *loss, float *lse, float *workspace, int64_t n_workspace, void *stream)
{
    const zero_status st = zs::xent_forward_check(rows, vocab, hidden, x, ldx, w, ldw, w_order, targets, loss, lse,
                                                  workspace, n_workspace);
    if (st != ZERO_OK)
        return st;
    return zs::xent_forward_run(rows, vocab, hidden, x, ldx, w, ldw, w_order, targets, loss, lse, workspace,
                                static_cast<hipStream_t>(stream));
}

zero_status zero_linear_xent_backward(int64_t rows, int64_t vocab, int64_t hidden, const uint16_t *x, int64_t ldx,
                                      const uint16_t *w, int64_t ldw, int32_t w_order, const int64_t *targets,
                                      const float *lse, const float *dloss, void *dx, int64_t lddx,
                                      int32_t dx_dtype, void *dw, int64_t lddw, int32_t dw_dtype, int64_t piece,
                                      float *workspace, int64_t n_workspace, void *stream)
{
    const zero_status st = zs::xent_backward_check(rows, vocab, hidden, x, ldx, w, ldw, w_order, targets, lse, dloss,
                                                   dx, lddx, dx_dtype, dw, lddw, dw_dtype, piece, workspace,
                                                   n_workspace);
    if (st != ZERO_OK)
        return st;
    return zs::xent_backward_run(rows, vocab, hidden, x, ldx, w, ldw, w_order, targets, lse, dloss, dx, lddx, dx_dtype,
                                 dw, lddw, dw_dtype, piece, workspace, static_cast<hipStream_t>(stream));
}

}  // extern "C"
