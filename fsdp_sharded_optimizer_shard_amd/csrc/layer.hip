// What a linear layer does around its product: the product with bias,
// activation and residual in its epilogue, the gradient of that epilogue,
// activations kept in 8 bits for the backward pass, and products grouped by
// expert.  The products run on the tiles of gemm_tile.h and on two more for
// shapes that those leave to a part of the CUs.
//
// All of them compute in fp32 from bf16 operands and leave through one
// epilogue, LayerEpi; which tile a product takes depends on its sizes and on
// how its operands are stored, and is decided where it is launched, with what
// was measured on both sides.
#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>
#include <type_traits>

#include "act.h"
#include "checks.h"
#include "gemm_tile.h"
#include "gemm_place.h"
#include "products.h"
#include "vec.h"

namespace zs {

namespace {

// -------------------------------------------------------- the epilogue --

struct EpiArgs {
    void *C;
    const void *bias, *residual;
    void *z;           // kept pre-activation: bf16, or codes when z_scales is set
    uint8_t *z_scales;
    uint8_t *o, *o_scales;  // C kept in 8 bits
    int64_t ldc, ldr, ldz, ldzs, ldo, ldos;
    int32_t act;
    bool c_bf16, bias_bf16, r_bf16;
    bool vec;  // 16-byte aligned rows in every matrix but the checkpoints
};

// y = act(z) + residual with z = sum + bias, on the way from a wave's
// accumulators to memory.  32 rows of the wave's tile at a time go through
// its own corner of LDS (the K loop is done with it): the accumulators are
// column-striped over lanes, memory wants whole rows, and the 8-bit code
// wants whole columns of 32 rows -- which these 32 rows are, as every tile
// begins at a multiple of 32 rows of C.  Rows in LDS are CW + 4 floats long,
// so that the row pass's 16-byte reads of neighbouring rows interleave over
// the banks.
struct LayerEpi {
    const EpiArgs &p;
    ZS_LDS float *lds;  // 32 * (CW + 4) floats of this wave

    // Codes of 32 rows x CW columns held in LDS, blocks along rows.  Lane:
    // 4 columns of 32 / RG rows.
    template <int CW>
    __device__ __forceinline__ void encode(uint8_t *codes, int64_t ld, uint8_t *scales, int64_t lds_,
                                           int64_t row0, int64_t col0, int64_t M, int64_t N,
                                           int lane) const
    {
        constexpr int Q = CW / 4, RG = 64 / Q, R = 32 / RG;
        const int quad = lane % Q, rg = lane / Q;
        const int64_t col = col0 + 4 * quad, row = row0 + rg * R;
        float x[R][4];
        uint32_t mx[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const f32x4 v = *reinterpret_cast<const ZS_LDS f32x4 *>(lds + (rg * R + i) * (CW + 4) + 4 * quad);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[i][k] = v[k];
                const uint32_t m = row + i < M ? mag_bits(v[k]) : 0u;
                mx[k] = m > mx[k] ? m : mx[k];
            }
        }
#pragma unroll
        for (int s = Q; s < 64; s *= 2)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t m = (uint32_t)__shfl_xor((int)mx[k], s, 64);
                mx[k] = m > mx[k] ? m : mx[k];
            }
        const int n = (int)(N - col < 4 ? N - col : 4);
        if (n <= 0)
            return;
        float inv[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t b = block_byte(mx[k]);
            inv[k] = inv_scale(b);
            if (rg == 0 && k < n && row0 < M)
                scales[(row0 >> 5) * lds_ + col + k] = (uint8_t)b;
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (row + i >= M)
                break;
            const uint32_t w = code4(coder_in(x[i][0]) * inv[0], coder_in(x[i][1]) * inv[1],
                                     coder_in(x[i][2]) * inv[2], coder_in(x[i][3]) * inv[3]);
            uint8_t *q = codes + (row + i) * ld + col;
            if (n == 4) {
                *reinterpret_cast<uint32_t *>(q) = w;
            } else {
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    if (k < n)
                        q[k] = (uint8_t)(w >> (8 * k));
            }
        }
    }

    __device__ __forceinline__ float bf16_at(const void *q, int64_t i) const
    {
        return __uint_as_float((uint32_t)static_cast<const uint16_t *>(q)[i] << 16);
    }

    // Eight residual values as loaded: bf16 in lo, fp32 in lo and hi.
    struct Res {
        uint4 lo, hi;
    };
    __device__ __forceinline__ Res load_residual(int64_t i) const
    {
        Res r = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (p.r_bf16) {
            r.lo = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.residual) + i);
        } else {
            r.lo = *reinterpret_cast<const uint4 *>(static_cast<const float *>(p.residual) + i);
            r.hi = *reinterpret_cast<const uint4 *>(static_cast<const float *>(p.residual) + i + 4);
        }
        return r;
    }

    // 32 whole rows x CW columns with every access 16 bytes: RPI rows a pass,
    // a lane's 8 columns of one.  The passes are a loop, so that the epilogue
    // stays a few KB of code (unrolled, its 28000 instructions cost more than
    // they did), and the residual is fetched one pass ahead.
    template <int CW, int ACT>
    __device__ __forceinline__ void rows_fast(int64_t row0, int64_t col0, Res next, int lane) const
    {
        constexpr int LPR = CW / 8, RPI = 64 / LPR, NP = 32 / RPI;
        int64_t row = row0 + lane / LPR;
        const int64_t col = col0 + 8 * (lane % LPR);
        ZS_LDS float *l = lds + (lane / LPR) * (CW + 4) + 8 * (lane % LPR);
#pragma unroll 1
        for (int it = 0; it < NP; ++it, row += RPI, l += RPI * (CW + 4)) {
            const Res cur = next;
            if (p.residual && it + 1 < NP)
                next = load_residual((row + RPI) * p.ldr + col);
            ZS_LDS f32x4 *q = reinterpret_cast<ZS_LDS f32x4 *>(l);
            const f32x4 lo = q[0], hi = q[1];
            float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            if (p.z && !p.z_scales)
                store8(p.z, true, row * p.ldz + col, true, 8, x);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] = act<ACT>(x[k]);
            if (p.residual) {
                float y[8];
                if (p.r_bf16) {
                    widen8(cur.lo, y);
                } else {
                    const uint32_t w[8] = {cur.lo.x, cur.lo.y, cur.lo.z, cur.lo.w,
                                           cur.hi.x, cur.hi.y, cur.hi.z, cur.hi.w};
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        y[k] = __uint_as_float(w[k]);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    x[k] += y[k];
            }
            store8(p.C, p.c_bf16, row * p.ldc + col, true, 8, x);
            if (p.o) {
                if (p.c_bf16)
                    widen8(make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                                      pack_bf16(x[6], x[7])),
                           x);
                q[0] = f32x4{x[0], x[1], x[2], x[3]};
                q[1] = f32x4{x[4], x[5], x[6], x[7]};
            }
        }
    }

    // The same element by element, for edges and unaligned matrices; a wave
    // still covers neighbouring columns.
    template <int CW>
    __device__ __forceinline__ void rows_slow(int64_t row0, int64_t col0, int64_t M, int64_t N, int lane) const
    {
#pragma unroll 1
        for (int e = lane; e < 32 * CW; e += 64) {
            const int r = e / CW, c = e % CW;
            const int64_t row = row0 + r, col = col0 + c;
            if (row >= M || col >= N)
                continue;
            float x = lds[r * (CW + 4) + c];
            if (p.z && !p.z_scales)
                static_cast<uint16_t *>(p.z)[row * p.ldz + col] = (uint16_t)pack_bf16(x, x);
            by_act(p.act, [&](auto a) { x = act<decltype(a)::value>(x); });
            if (p.residual)
                x += p.r_bf16 ? bf16_at(p.residual, row * p.ldr + col)
                              : static_cast<const float *>(p.residual)[row * p.ldr + col];
            if (p.c_bf16) {
                const uint32_t h = pack_bf16(x, x);
                static_cast<uint16_t *>(p.C)[row * p.ldc + col] = (uint16_t)h;
                x = __uint_as_float(h << 16);
            } else {
                static_cast<float *>(p.C)[row * p.ldc + col] = x;
            }
            if (p.o)
                lds[r * (CW + 4) + c] = x;
        }
    }

    template <int CW>
    __device__ __forceinline__ bool whole_rows(int64_t row0, int64_t col0, int64_t M, int64_t N) const
    {
        return p.vec && row0 + 32 <= M && col0 + CW <= N;
    }

    template <int CW>
    __device__ __forceinline__ Res first_residual(int64_t row0, int64_t col0, int64_t M, int64_t N,
                                                  int lane) const
    {
        if (!p.residual || !whole_rows<CW>(row0, col0, M, N))
            return Res{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        return load_residual((row0 + lane / (CW / 8)) * p.ldr + col0 + 8 * (lane % (CW / 8)));
    }

    // z of 32 rows x CW columns is in LDS.
    template <int CW>
    __device__ __forceinline__ void rows32(int64_t row0, int64_t col0, int64_t M, int64_t N, Res first,
                                           int lane) const
    {
        wave_lds_order();
        if (row0 >= M || col0 >= N)
            return;
        if (p.z_scales)
            encode<CW>(static_cast<uint8_t *>(p.z), p.ldz, p.z_scales, p.ldzs, row0, col0, M, N, lane);
        if (whole_rows<CW>(row0, col0, M, N))
            by_act(p.act, [&](auto a) { rows_fast<CW, decltype(a)::value>(row0, col0, first, lane); });
        else
            rows_slow<CW>(row0, col0, M, N, lane);
        // C in 8 bits is coded from C as stored, so it is what coding C
        // afterwards would give.
        if (p.o) {
            wave_lds_order();
            encode<CW>(p.o, p.ldo, p.o_scales, p.ldos, row0, col0, M, N, lane);
        }
        wave_lds_order();
    }

    // The bias of TN columns W apart, the loads side by side.
    template <int TN, int W>
    __device__ __forceinline__ void load_bias(int64_t col, int64_t N, float (&b)[TN]) const
    {
#pragma unroll
        for (int j = 0; j < TN; ++j)
            b[j] = 0.0f;
        if (!p.bias)
            return;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int64_t c = col + W * j < N ? col + W * j : N - 1;
            b[j] = p.bias_bf16 ? bf16_at(p.bias, c) : static_cast<const float *>(p.bias)[c];
        }
    }

    // Rows 32 I .. of the wave's tile; by recursion, so that every accumulator
    // index is a constant whatever the unroller thinks of the body.
    template <int I, int TM, int TN>
    __device__ __forceinline__ void step32(const f32x16 (&acc)[TM][TN], const float (&b)[TN], int64_t row0,
                                           int64_t col0, int64_t M, int64_t N, int lane) const
    {
        if constexpr (I < TM) {
            constexpr int CW = 32 * TN;
            const int fr = lane & 31, fh = lane >> 5;
            const Res first = first_residual<CW>(row0 + 32 * I, col0, M, N, lane);
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    lds[(8 * (v >> 2) + 4 * fh + (v & 3)) * (CW + 4) + 32 * j + fr] = acc[I][j][v] + b[j];
            rows32<CW>(row0 + 32 * I, col0, M, N, first, lane);
            step32<I + 1>(acc, b, row0, col0, M, N, lane);
        }
    }

    template <int I, int TM, int TN>
    __device__ __forceinline__ void step16(const f32x4 (&acc)[TM][TN], const float (&b)[TN], int64_t row0,
                                           int64_t col0, int64_t M, int64_t N, int lane) const
    {
        if constexpr (I < TM) {
            constexpr int CW = 16 * TN;
            const int r16 = lane & 15, g = lane >> 4;
            const Res first = first_residual<CW>(row0 + 16 * I, col0, M, N, lane);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        lds[(16 * h + 4 * g + v) * (CW + 4) + 16 * j + r16] = acc[I + h][j][v] + b[j];
            rows32<CW>(row0 + 16 * I, col0, M, N, first, lane);
            step16<I + 2>(acc, b, row0, col0, M, N, lane);
        }
    }

    template <int TM, int TN>
    __device__ __forceinline__ void tile32(const f32x16 (&acc)[TM][TN], int64_t row0, int64_t col0,
                                           int64_t M, int64_t N, int lane) const
    {
        float b[TN];
        load_bias<TN, 32>(col0 + (lane & 31), N, b);
        __syncthreads();  // every wave is done with the K loop's LDS
        step32<0>(acc, b, row0, col0, M, N, lane);
    }

    template <int TM, int TN>
    __device__ __forceinline__ void tile16(const f32x4 (&acc)[TM][TN], int64_t row0, int64_t col0,
                                           int64_t M, int64_t N, int lane) const
    {
        float b[TN];
        load_bias<TN, 16>(col0 + (lane & 15), N, b);
        __syncthreads();
        step16<0>(acc, b, row0, col0, M, N, lane);
    }
};

// ------------------------------------------------------ product kernels --

template <int BM, int BN, bool A_KOUTER, bool B_KOUTER>
__global__ __launch_bounds__(kGT) void epi_kernel(int64_t M, int64_t N, int64_t K,
                                                  const uint16_t *__restrict__ A, int64_t lda,
                                                  const uint16_t *__restrict__ B, int64_t ldb,
                                                  EpiArgs args, int tiles_m, int tiles_n, int n_big)
{
    ZS_STAGES(BM, BN);
    const LayerEpi epi{args, ZS_CORNER};
    int64_t m0, n0;
    if (place<BM, BN>(tiles_m, tiles_n, n_big, m0, n0))
        gemm_tile<BM, BN, A_KOUTER, B_KOUTER>(M, N, K, A, lda, B, ldb, epi, m0, n0, As, Bs);
    else if constexpr (BM == kBM)
        gemm_tile<BM / 2, BN, A_KOUTER, B_KOUTER>(M, N, K, A, lda, B, ldb, epi, m0, n0, As, Bs);
}

// X W on 256 x 256 tiles and their halves.
#define ZS_AP                                                                                      \
    __shared__ __attribute__((aligned(1024))) char pa0[kPair], pa1[kPair];                         \
    __shared__ __attribute__((aligned(1024))) char b0[kStage], b1[kStage], b2[kStage], b3[kStage]; \
    ZS_LDS char *const Bs[kStages] = {(ZS_LDS char *)b0, (ZS_LDS char *)b1, (ZS_LDS char *)b2,     \
                                      (ZS_LDS char *)b3};                                          \
    const LayerEpi epi{args, corner((ZS_LDS char *)pa0, (ZS_LDS char *)pa0 + kPair / 2,            \
                                    (ZS_LDS char *)pa1, (ZS_LDS char *)pa1 + kPair / 2,            \
                                    (ZS_LDS char *)b0, (ZS_LDS char *)b1, (ZS_LDS char *)b2,       \
                                    (ZS_LDS char *)b3)}

__global__ __launch_bounds__(kGT) void epi_kernel_ap(int64_t M, int64_t N, int64_t K,
                                                     const uint16_t *__restrict__ A, int64_t lda,
                                                     const uint16_t *__restrict__ B, int64_t ldb,
                                                     EpiArgs args, int tiles_m, int tiles_n, int n_big)
{
    ZS_AP;
    int64_t m0, n0;
    if (place<kBM, kBN>(tiles_m, tiles_n, n_big, m0, n0))
        gemm_tile_ap<kBM>(M, N, K, A, lda, B, ldb, epi, m0, n0, (ZS_LDS char *)pa0, (ZS_LDS char *)pa1, Bs);
    else
        gemm_tile_ap<kBM / 2>(M, N, K, A, lda, B, ldb, epi, m0, n0, (ZS_LDS char *)pa0, (ZS_LDS char *)pa1,
                              Bs);
}

template <int BM, int BN>
__global__ __launch_bounds__(kGT) void epi_kernel_kp(int64_t M, int64_t N, int64_t K,
                                                     const uint16_t *__restrict__ A, int64_t lda,
                                                     const uint16_t *__restrict__ B, int64_t ldb,
                                                     EpiArgs args, int tiles_m, int tiles_n, int n_big)
{
    ZS_PAIRS(BM, BN);
    const LayerEpi epi{args, ZS_CORNER_KP((BM < BN ? BM : BN) * 64)};
    int64_t m0, n0;
    if (place<BM, BN>(tiles_m, tiles_n, n_big, m0, n0))
        gemm_tile_kp<BM, BN>(M, N, K, A, lda, B, ldb, epi, m0, n0, ZS_P);
    else if constexpr (BM == kBM)
        gemm_tile_kp<BM / 2, BN>(M, N, K, A, lda, B, ldb, epi, m0, n0, ZS_P);
}

// ------------------------------------------------- few tiles, long sums --

// A 128 x 128 tile for products that have too few tiles to fill the CUs with
// 256 x 256 ones, so that a CU runs one block: the two halves of its waves
// take alternate K tiles of 32, each half a 2 x 2 grid of 64 x 64, and add
// their sums at the end.  Against the 2 x 4 grid of gemm_tile on one K tile
// at a time, a barrier stands between twice the products and a fragment
// serves twice as many.  1000 x 4096 x 14336 (256 tiles, every block alone on
// its CU): 153 -> 126 us with a K-outer B, 203 -> 139 with a K-inner one.  What
// bounds it then is the fetch of operands that no other block shares, some 60
// GB/s a CU: 141 us with 64-byte rows of a K-inner operand, 126 with 128.
//
// Stage g % 4 holds K tiles 2 g and 2 g + 1 of both operands, 16 KB each, A
// first; half h of the waves reads tile 2 g + h.  A K-outer operand's tiles lie
// one after the other, each fetched by the waves that read it; a K-inner
// operand is one 64-k pair in gemm_tile_kp's layout, fetched by all waves in
// whole 128-byte rows.  A K tile past the last reads as zeros.
constexpr int kTwo = 2 * 128 * kBK * 2;  // bytes of one operand's two tiles

template <bool A_KOUTER, bool B_KOUTER, class Epi>
__device__ __forceinline__ void gemm_tile_k2(int64_t M, int64_t N, int64_t K,
                                             const uint16_t *__restrict__ A, int64_t lda,
                                             const uint16_t *__restrict__ B, int64_t ldb, const Epi &epi,
                                             int64_t m0, int64_t n0, ZS_LDS char *const (&Ss)[kStages],
                                             ZS_LDS float *mine, ZS_LDS float *partner)
{
    constexpr int BM = 128, BN = 128, TM = 2, TN = 2, NF = TM + TN, NMF = TM * TN;
    constexpr int NRD = TM * Op<BM, A_KOUTER>::NRD + TN * Op<BN, B_KOUTER>::NRD;
    constexpr int NI = 2, D = 2 * NI;  // loads of one operand, of both, per wave and stage

    const int t = threadIdx.x, lane = t & 63, w8 = __builtin_amdgcn_readfirstlane(t >> 6);
    const int half = w8 >> 2, wave = w8 & 3;
    const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;

    uint32_t va[NI], vb[NI];
    int ka[NI];
#pragma unroll
    for (int n = 0; n < NI; ++n) {
        va[n] = A_KOUTER ? dma_offset<BM, true>(lda, wave + 4 * n, lane, 0) : kp_dma_offset(lda, w8, lane, n);
        vb[n] = B_KOUTER ? dma_offset<BN, true>(ldb, wave + 4 * n, lane, 0) : kp_dma_offset(ldb, w8, lane, n);
        ka[n] = kp_kofs(w8, lane, n);
    }
    auto frag_at = [&](auto outer, int w0, int s) {
        if constexpr (decltype(outer)::value)
            return half * (kTwo / 2) + frag_offset<128, true>(w0, s, lane);
        else
            return kp_pos(w0 + (lane & 31), 4 * half + 2 * s + (lane >> 5));
    };
    int fa_off[TM][2], fb_off[TN][2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
            fa_off[i][s] = frag_at(IC<A_KOUTER>{}, wm + 32 * i, s);
#pragma unroll
        for (int j = 0; j < TN; ++j)
            fb_off[j][s] = kTwo + frag_at(IC<B_KOUTER>{}, wn + 32 * j, s);
    }

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v)
                acc[i][j][v] = 0.0f;

    const int64_t g_n = (K + 2 * kBK - 1) / (2 * kBK), g_full = K / (2 * kBK);
    auto dma = [&](auto st, auto whole, int64_t g) {
        constexpr int S = decltype(st)::value;
        constexpr bool WHOLE = decltype(whole)::value != 0;
        const int64_t k0 = 2 * g * kBK, kh = k0 + half * kBK;
        const __amdgpu_buffer_rsrc_t ra = A_KOUTER ? rsrc(A + kh * lda + m0, ((K - 1 - kh) * lda + M - m0) * 2)
                                                   : rsrc(A + m0 * lda + k0, ((M - 1 - m0) * lda + K - k0) * 2);
        const __amdgpu_buffer_rsrc_t rb = B_KOUTER ? rsrc(B + kh * ldb + n0, ((K - 1 - kh) * ldb + N - n0) * 2)
                                                   : rsrc(B + n0 * ldb + k0, ((N - 1 - n0) * ldb + K - k0) * 2);
#pragma unroll
        for (int n = 0; n < NI; ++n) {
            const uint32_t o = !WHOLE && !A_KOUTER && k0 + ka[n] >= K ? kOOB : va[n];
            ZS_LDS char *d = Ss[S] + (A_KOUTER ? half * (kTwo / 2) + (wave + 4 * n) * 1024 : (w8 + 8 * n) * 1024);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (ZS_LDS void *)d, 16, o, 0, 0, 0);
        }
#pragma unroll
        for (int n = 0; n < NI; ++n) {
            const uint32_t o = !WHOLE && !B_KOUTER && k0 + ka[n] >= K ? kOOB : vb[n];
            ZS_LDS char *d = Ss[S] + kTwo +
                             (B_KOUTER ? half * (kTwo / 2) + (wave + 4 * n) * 1024 : (w8 + 8 * n) * 1024);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (ZS_LDS void *)d, 16, o, 0, 0, 0);
        }
    };
    bf16x8 fa0[TM], fb0[TN], fa1[TM], fb1[TN];
    auto frags = [&](auto st, int s, bf16x8 (&fa)[TM], bf16x8 (&fb)[TN]) {
        constexpr int S = decltype(st)::value;
#pragma unroll
        for (int i = 0; i < TM; ++i)
            fa[i] = frag_read<BM, A_KOUTER>(Ss[S], fa_off[i][s]);
#pragma unroll
        for (int j = 0; j < TN; ++j)
            fb[j] = frag_read<BN, B_KOUTER>(Ss[S], fb_off[j][s]);
    };
    auto mma = [&](const bf16x8 (&fa)[TM], const bf16x8 (&fb)[TN], int lo, int hi) {
#pragma unroll
        for (int q = 0; q < NMF; ++q)
            if (q >= lo && q < hi)
                acc[q / TN][q % TN] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                    fa[q / TN], fb[q % TN], acc[q / TN][q % TN], 0, 0, 0);
    };
    auto wait_for = [&](int64_t g1) {
        const int64_t after = g_n - 1 - g1;
        if (after >= 2)
            wait_vm_lgkm0<2 * D>();
        else if (after == 1)
            wait_vm_lgkm0<D>();
        else
            wait_vm_lgkm0<0>();
    };
    // Pair of K tiles g, as gemm_tile's tile.
    auto tile = [&](auto st, auto steady, int64_t g) {
        constexpr int S = decltype(st)::value;
        constexpr bool STEADY = decltype(steady)::value != 0;
        constexpr int SN = (S + kStages - 1) % kStages, S1 = (S + 1) % kStages;
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (STEADY)
            dma(IC<SN>{}, IC<1>{}, g + kStages - 1);
        else if (g + kStages - 1 < g_n)
            dma(IC<SN>{}, IC<0>{}, g + kStages - 1);
        frags(IC<S>{}, 1, fa1, fb1);
        mma(fa0, fb0, 0, NMF);
        seq<NF, NMF, NRD, STEADY ? D : 0>();
        mma(fa1, fb1, 0, NMF / 2);
        __builtin_amdgcn_sched_group_barrier(0x008, NMF / 2, 0);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (STEADY)
            wait_vm_lgkm0<2 * D>();
        else
            wait_for(g + 1);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        if (STEADY || g + 1 < g_n)
            frags(IC<S1>{}, 0, fa0, fb0);
        mma(fa1, fb1, NMF / 2, NMF);
        seq<NF, NMF / 2, NRD, 0>();
    };
    if (g_n > 0) {
        dma(IC<0>{}, IC<0>{}, 0);
        if (g_n > 1)
            dma(IC<1>{}, IC<0>{}, 1);
        if (g_n > 2)
            dma(IC<2>{}, IC<0>{}, 2);
        wait_for(0);
        __builtin_amdgcn_s_barrier();
        frags(IC<0>{}, 0, fa0, fb0);
        int64_t g = 0;
        for (; g + 2 * kStages - 1 <= g_full; g += kStages) {
            tile(IC<0>{}, IC<1>{}, g);
            tile(IC<1>{}, IC<1>{}, g + 1);
            tile(IC<2>{}, IC<1>{}, g + 2);
            tile(IC<3>{}, IC<1>{}, g + 3);
        }
        for (; g < g_n; g += kStages) {
            tile(IC<0>{}, IC<0>{}, g);
            if (g + 1 < g_n)
                tile(IC<1>{}, IC<0>{}, g + 1);
            if (g + 2 < g_n)
                tile(IC<2>{}, IC<0>{}, g + 2);
            if (g + 3 < g_n)
                tile(IC<3>{}, IC<0>{}, g + 3);
        }
    }
    // Wave (wave, half) hands its partner the rows 32 (1 - half) .. and keeps
    // the others: the sum of the even K tiles plus that of the odd ones.
    __syncthreads();
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v)
            partner[(16 * j + v) * 64 + lane] = half ? acc[0][j][v] : acc[1][j][v];
    __syncthreads();
    f32x16 sum[1][TN];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            const float other = mine[(16 * j + v) * 64 + lane];
            sum[0][j][v] = half ? other + acc[1][j][v] : acc[0][j][v] + other;
        }
    epi.template tile32<1, TN>(sum, m0 + wm + 32 * half, n0 + wn, M, N, lane);
}

template <bool A_KOUTER, bool B_KOUTER>
__global__ __launch_bounds__(kGT) void epi_kernel_k2(int64_t M, int64_t N, int64_t K,
                                                     const uint16_t *__restrict__ A, int64_t lda,
                                                     const uint16_t *__restrict__ B, int64_t ldb,
                                                     EpiArgs args, int tiles_m, int tiles_n)
{
    __shared__ __attribute__((aligned(1024))) char s0[2 * kTwo], s1[2 * kTwo],
        s2[2 * kTwo], s3[2 * kTwo];
    ZS_LDS char *const Ss[kStages] = {(ZS_LDS char *)s0, (ZS_LDS char *)s1, (ZS_LDS char *)s2,
                                      (ZS_LDS char *)s3};
#define ZS_S(n) (ZS_LDS char *)s##n, (ZS_LDS char *)s##n + kTwo
    ZS_LDS float *mine = corner(ZS_S(0), ZS_S(1), ZS_S(2), ZS_S(3));
    ZS_LDS float *partner = corner(ZS_S(2), ZS_S(3), ZS_S(0), ZS_S(1));
#undef ZS_S
    const LayerEpi epi{args, mine};
    int64_t m0, n0;
    place<128, 128>(tiles_m, tiles_n, tiles_m * tiles_n, m0, n0);
    gemm_tile_k2<A_KOUTER, B_KOUTER>(M, N, K, A, lda, B, ldb, epi, m0, n0, Ss, mine, partner);
}

// ------------------------------------------------------------- few rows --

// 32 x 32 tiles for products of few rows, where the weights' bytes are the
// work and 128 x 128 tiles would leave most CUs without a block: K is split
// over the block's eight waves, 64 k at a time, each wave with two stages of
// LDS and loads of its own and no barrier until the sums meet.  A stage of
// the 32 A rows, or of 32 rows of a K-inner B, is gemm_tile_kp's pair (128-byte
// rows, swizzled); of a K-outer B it is 64 k rows of 64 bytes as they come: the
// transposing reads of a half wave take four whole rows, 256 bytes, so they
// fall on all banks once.  Up to two stages, 128 KB a CU, are in flight.
constexpr int kSkM = 32, kSkN = 32, kSkK = 64;
constexpr int kSkOp = 32 * 128;  // bytes of one operand's stage of one wave

template <bool B_KOUTER>
__device__ __forceinline__ void skinny_tile(int64_t M, int64_t N, int64_t K, const uint16_t *__restrict__ A,
                                            int64_t lda, const uint16_t *__restrict__ B, int64_t ldb,
                                            const EpiArgs &args, int64_t m0, int64_t n0)
{
    __shared__ __attribute__((aligned(1024))) char s0[kNW * 2 * kSkOp], s1[kNW * 2 * kSkOp];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 31, fh = lane >> 5;
    auto stage = [&](auto st) -> ZS_LDS char * {
        if constexpr (decltype(st)::value == 0)
            return (ZS_LDS char *)s0 + wave * 2 * kSkOp;
        else
            return (ZS_LDS char *)s1 + wave * 2 * kSkOp;
    };

    // A's loads of eight rows; rows past M hold what LDS held and end in rows of
    // C past M.
    const int na = M - m0 >= 32 ? 4 : (int)((M - m0 + 7) / 8);
    uint32_t va[4], vb[4];
    int ka[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        va[n] = kp_dma_offset(lda, n, lane, 0);
        ka[n] = kp_kofs(n, lane, 0);
        vb[n] = B_KOUTER ? (uint32_t)(((16 * n + (lane >> 2)) * ldb + 8 * (lane & 3)) * 2)
                         : kp_dma_offset(ldb, n, lane, 0);
    }
    // K tile t of 64 into a stage.
    auto dma = [&](auto st, int64_t t) {
        const int64_t k0 = t * kSkK;
        const __amdgpu_buffer_rsrc_t ra = rsrc(A + m0 * lda + k0, ((M - 1 - m0) * lda + K - k0) * 2);
        const __amdgpu_buffer_rsrc_t rb = B_KOUTER ? rsrc(B + k0 * ldb + n0, ((K - 1 - k0) * ldb + N - n0) * 2)
                                                   : rsrc(B + n0 * ldb + k0, ((N - 1 - n0) * ldb + K - k0) * 2);
        ZS_LDS char *d = stage(st);
#pragma unroll
        for (int n = 0; n < 4; ++n)
            if (n < na)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (ZS_LDS void *)(d + n * 1024), 16,
                                                         k0 + ka[n] >= K ? kOOB : va[n], 0, 0, 0);
#pragma unroll
        for (int n = 0; n < 4; ++n)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (ZS_LDS void *)(d + kSkOp + n * 1024), 16,
                                                     !B_KOUTER && k0 + ka[n] >= K ? kOOB : vb[n], 0, 0, 0);
    };
    f32x16 acc;
#pragma unroll
    for (int v = 0; v < 16; ++v)
        acc[v] = 0.0f;
    auto step = [&](auto st, int64_t t, int64_t t_n) {
        const ZS_LDS char *d = stage(st);
        // the other stage's na + 4 loads may stay in flight
        if (t + kNW >= t_n)
            wait_vm_lgkm0<0>();
        else if (na == 4)
            wait_vm_lgkm0<8>();
        else if (na == 3)
            wait_vm_lgkm0<7>();
        else if (na == 2)
            wait_vm_lgkm0<6>();
        else
            wait_vm_lgkm0<5>();
        bf16x8 fa[4], fb[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            fa[s] = *reinterpret_cast<const ZS_LDS bf16x8 *>(d + kp_pos(fr, 2 * s + fh));
            if (!B_KOUTER) {
                fb[s] = *reinterpret_cast<const ZS_LDS bf16x8 *>(d + kSkOp + kp_pos(fr, 2 * s + fh));
            } else {
                const int j = lane & 15, kr = 16 * s + 8 * fh + (j >> 2);
                const int o = kr * 64 + 32 * ((lane >> 4) & 1) + 8 * (j & 3);
                const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZS_LDS s16x4 *)(d + kSkOp + o));
                const s16x4 hi =
                    __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZS_LDS s16x4 *)(d + kSkOp + o + 4 * 64));
                const s16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                fb[s] = __builtin_bit_cast(bf16x8, v);
            }
        }
        // The stage is overwritten only after every read of it has returned.
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0) alone
        __builtin_amdgcn_sched_barrier(0);
        if (t + 2 * kNW < t_n)
            dma(st, t + 2 * kNW);
#pragma unroll
        for (int s = 0; s < 4; ++s)
            acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[s], fb[s], acc, 0, 0, 0);
    };
    const int64_t t_n = (K + kSkK - 1) / kSkK;
    if (wave < t_n)
        dma(IC<0>{}, wave);
    if (wave + kNW < t_n)
        dma(IC<1>{}, wave + kNW);
    for (int64_t t = wave; t < t_n; t += 2 * kNW) {
        step(IC<0>{}, t, t_n);
        if (t + kNW < t_n)
            step(IC<1>{}, t + kNW, t_n);
    }
    // The eight sums, added in the waves' order: 4 KB a wave, each wave adding
    // two of the sixteen accumulators.
    __syncthreads();
    ZS_LDS float *part = (ZS_LDS float *)(ZS_LDS char *)s0;
#pragma unroll
    for (int v = 0; v < 16; ++v)
        part[(wave * 16 + v) * 64 + lane] = acc[v];
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int v = 2 * wave + q;
        float s = part[v * 64 + lane];
#pragma unroll
        for (int w = 1; w < kNW; ++w)
            s += part[(w * 16 + v) * 64 + lane];
        part[v * 64 + lane] = s;
    }
    __syncthreads();
    f32x16 sum[1][1];
#pragma unroll
    for (int v = 0; v < 16; ++v)
        sum[0][0][v] = part[v * 64 + lane];
    // The first wave stores; for the others the tile lies past the last row.
    const LayerEpi epi{args, (ZS_LDS float *)((ZS_LDS char *)s1 + wave * 2 * kSkOp)};
    epi.tile32<1, 1>(sum, wave == 0 ? m0 : M, n0, M, N, lane);
}

// The same for a K-outer B of many columns: 64 of them, so that its k rows come
// in whole 128-byte lines, 32 k at a time, three stages a wave (6 KB each, 144 KB
// a CU).  A's rows lie as in gemm_tile's 32-k stage; the 64-byte half h of B's k
// row r sits at h ^ ((r >> 1) & 1), so that the four rows a half wave reads at
// once fall on all banks.  1 x 14336 x 4096: 27 us, 4.3 TB/s of weights, against 37
// in 32 columns; 32 rows 31 and 42, 64 x 8192 x 8192 46 and 60, 128 x 4096 x 4096 16
// and 21.  With fewer blocks than that makes, 32 columns keep more CUs loading: 1
// x 4096 x 14336 (64 blocks) 60 and 54, 64 x 4096 x 4096 (128) 16.1 and 13.4, 1 x
// 8192 x 28672 (128) 125 and 113.
constexpr int kOuN = 64, kOuStages = 3;
constexpr int kOuA = 32 * kBK * 2, kOuStage = kOuA + kBK * kOuN * 2;  // bytes of one wave

__device__ __forceinline__ void skinny_outer_tile(int64_t M, int64_t N, int64_t K,
                                                  const uint16_t *__restrict__ A, int64_t lda,
                                                  const uint16_t *__restrict__ B, int64_t ldb,
                                                  const EpiArgs &args, int64_t m0, int64_t n0)
{
    __shared__ __attribute__((aligned(1024))) char s0[kNW * kOuStage], s1[kNW * kOuStage], s2[kNW * kOuStage];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 31, fh = lane >> 5;
    auto stage = [&](auto st) -> ZS_LDS char * {
        if constexpr (decltype(st)::value == 0)
            return (ZS_LDS char *)s0 + wave * kOuStage;
        else if constexpr (decltype(st)::value == 1)
            return (ZS_LDS char *)s1 + wave * kOuStage;
        else
            return (ZS_LDS char *)s2 + wave * kOuStage;
    };

    // A's loads of sixteen rows; rows past M hold what LDS held and end in rows
    // of C past M.
    const int na = M - m0 > 16 ? 2 : 1;
    uint32_t va[2], vb[4];
    int ka[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        va[n] = dma_offset<128, false>(lda, n, lane, 0);
        ka[n] = dma_kofs(n, lane, 0);
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const int r = 8 * n + (lane >> 3), c = (lane & 7) ^ (((r >> 1) & 1) << 2);
        vb[n] = (uint32_t)((r * ldb + 8 * c) * 2);
    }
    // K tile t of 32 into a stage.
    auto dma = [&](auto st, int64_t t) {
        const int64_t k0 = t * kBK;
        const __amdgpu_buffer_rsrc_t ra = rsrc(A + m0 * lda + k0, ((M - 1 - m0) * lda + K - k0) * 2);
        const __amdgpu_buffer_rsrc_t rb = rsrc(B + k0 * ldb + n0, ((K - 1 - k0) * ldb + N - n0) * 2);
        ZS_LDS char *d = stage(st);
#pragma unroll
        for (int n = 0; n < 2; ++n)
            if (n < na)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (ZS_LDS void *)(d + n * 1024), 16,
                                                         k0 + ka[n] >= K ? kOOB : va[n], 0, 0, 0);
#pragma unroll
        for (int n = 0; n < 4; ++n)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (ZS_LDS void *)(d + kOuA + n * 1024), 16, vb[n], 0, 0,
                                                     0);
    };
    f32x16 acc[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v)
            acc[j][v] = 0.0f;
    const int64_t t_n = (K + kBK - 1) / kBK;
    auto step = [&](auto st, int64_t t) {
        const ZS_LDS char *d = stage(st);
        // the later stages' na + 4 loads each may stay in flight
        if (t + kNW >= t_n) {
            wait_vm_lgkm0<0>();
        } else if (t + 2 * kNW >= t_n) {
            if (na == 2)
                wait_vm_lgkm0<6>();
            else
                wait_vm_lgkm0<5>();
        } else {
            if (na == 2)
                wait_vm_lgkm0<12>();
            else
                wait_vm_lgkm0<10>();
        }
        bf16x8 fa[2], fb[2][2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            fa[s] = *reinterpret_cast<const ZS_LDS bf16x8 *>(d + ki_pos(fr, 2 * s + fh));
            const int j4 = lane & 15, kr = 16 * s + 8 * fh + (j4 >> 2);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int o = kr * 128 + 64 * (j ^ (j4 >> 3)) + 32 * ((lane >> 4) & 1) + 8 * (j4 & 3);
                const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZS_LDS s16x4 *)(d + kOuA + o));
                const s16x4 hi =
                    __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZS_LDS s16x4 *)(d + kOuA + o + 4 * 128));
                const s16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                fb[s][j] = __builtin_bit_cast(bf16x8, v);
            }
        }
        // The stage is overwritten only after every read of it has returned.
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0) alone
        __builtin_amdgcn_sched_barrier(0);
        if (t + kOuStages * kNW < t_n)
            dma(st, t + kOuStages * kNW);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[s], fb[s][j], acc[j], 0, 0, 0);
    };
    if (wave < t_n)
        dma(IC<0>{}, wave);
    if (wave + kNW < t_n)
        dma(IC<1>{}, wave + kNW);
    if (wave + 2 * kNW < t_n)
        dma(IC<2>{}, wave + 2 * kNW);
    for (int64_t t = wave; t < t_n; t += kOuStages * kNW) {
        step(IC<0>{}, t);
        if (t + kNW < t_n)
            step(IC<1>{}, t + kNW);
        if (t + 2 * kNW < t_n)
            step(IC<2>{}, t + 2 * kNW);
    }
    // The eight sums, added in the waves' order: 4 KB a wave and 32 columns, each
    // wave adding two of the sixteen accumulators of both.
    __syncthreads();
    ZS_LDS float *part0 = (ZS_LDS float *)(ZS_LDS char *)s0, *part1 = (ZS_LDS float *)(ZS_LDS char *)s1;
#pragma unroll
    for (int v = 0; v < 16; ++v) {
        part0[(wave * 16 + v) * 64 + lane] = acc[0][v];
        part1[(wave * 16 + v) * 64 + lane] = acc[1][v];
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int v = 2 * wave + q;
        float x = part0[v * 64 + lane], y = part1[v * 64 + lane];
#pragma unroll
        for (int w = 1; w < kNW; ++w) {
            x += part0[(w * 16 + v) * 64 + lane];
            y += part1[(w * 16 + v) * 64 + lane];
        }
        part0[v * 64 + lane] = x;
        part1[v * 64 + lane] = y;
    }
    __syncthreads();
    f32x16 sum[1][1];
#pragma unroll
    for (int v = 0; v < 16; ++v)
        sum[0][0][v] = wave & 1 ? part1[v * 64 + lane] : part0[v * 64 + lane];
    // Two waves store, 32 columns each; for the others the tile lies past the
    // last row.
    const LayerEpi epi{args, (ZS_LDS float *)((ZS_LDS char *)s2 + wave * kOuStage)};
    epi.tile32<1, 1>(sum, wave < 2 ? m0 : M, n0 + 32 * (wave & 1), M, N, lane);
}

template <int BN, bool B_KOUTER>
__global__ __launch_bounds__(kGT) void skinny_kernel(int64_t M, int64_t N, int64_t K,
                                                     const uint16_t *__restrict__ A, int64_t lda,
                                                     const uint16_t *__restrict__ B, int64_t ldb,
                                                     EpiArgs args, int tiles_m)
{
    const int b = xcd_order(blockIdx.x, gridDim.x);
    const int64_t m0 = (int64_t)(b % tiles_m) * kSkM, n0 = (int64_t)(b / tiles_m) * BN;
    if constexpr (BN == kOuN)
        skinny_outer_tile(M, N, K, A, lda, B, ldb, args, m0, n0);
    else
        skinny_tile<B_KOUTER>(M, N, K, A, lda, B, ldb, args, m0, n0);
}

// Group e's rows [lo, hi), kept inside [0, rows] whatever the array holds.
__device__ __forceinline__ void group_range(const int64_t *off, int e, int64_t rows, int64_t &lo, int64_t &hi)
{
    lo = off[e];
    hi = off[e + 1];
    lo = lo < 0 ? 0 : lo > rows ? rows : lo;
    hi = hi < lo ? lo : hi > rows ? rows : hi;
}

// Inclusive sum over the 64 lanes, in registers: within rows of 16 lanes, then
// rows 0 and 2 into 1 and 3, then the lower half into the upper.  (Six
// exchanges through LDS would cost more than the lookup's loads.)
__device__ __forceinline__ int lane_sum(int x)
{
#define ZS_DPP(CTRL, ROWS) x += __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xf, false)
    ZS_DPP(0x111, 0xf);  // row_shr:1
    ZS_DPP(0x112, 0xf);
    ZS_DPP(0x114, 0xf);
    ZS_DPP(0x118, 0xf);
    ZS_DPP(0x142, 0xa);  // row_bcast:15
    ZS_DPP(0x143, 0xc);  // row_bcast:31
#undef ZS_DPP
    return x;
}

// Tiles of BM rows of group c + lane (0 past the last), and their running sum
// over the lanes.
template <int BM>
__device__ __forceinline__ int lane_tiles(const int64_t *off, int n_groups, int c, int64_t rows, int &sum)
{
    const int lane = threadIdx.x & 63;
    int64_t lo = 0, hi = 0;
    if (c + lane < n_groups)
        group_range(off, c + lane, rows, lo, hi);
    const int t = (int)((uint64_t)(hi - lo + BM - 1) / BM);
    sum = lane_sum(t);
    return t;
}

struct Place {
    int e, tile, row_tiles;  // group, tile number in the group, its row tiles
    int half;                // -1: whole, or 0 / 1 of a tile split in two
};

// Which tile this block computes, looked up by every wave for itself.  Tiles
// are numbered group after group; each XCD takes a contiguous run of them, so
// that its L2 sees one stretch of weights, and a last wave of at most half
// the CUs is split into half tiles, as in the plain product -- only that the
// number of tiles is the device's to know.  The lookup is on every block's
// path: with 64-bit scans through LDS it cost 8 us a block.
template <int BM>
__device__ __forceinline__ bool find_tile(const int64_t *off, int n_groups, int64_t rows, int tiles_n, int cus,
                                          Place &p)
{
    int sum;
    int t = lane_tiles<BM>(off, n_groups, 0, rows, sum);
    int total = __builtin_amdgcn_readlane(sum, 63);
    for (int c = 64; c < n_groups; c += 64) {
        int more;
        lane_tiles<BM>(off, n_groups, c, rows, more);
        total += __builtin_amdgcn_readlane(more, 63);
    }
    const int T = total * tiles_n, b = blockIdx.x, rem = (int)((unsigned)T % (unsigned)cus);
    const int whole = BM == kBM && rem <= cus / 2 ? T - rem : T;
    const int blocks = whole + 2 * (T - whole);
    if (b >= blocks)
        return false;
    int want;
    if (b < whole) {
        want = xcd_order(b, whole);
        p.half = -1;
    } else {
        const int h = xcd_order(b - whole, blocks - whole);
        want = whole + h / 2;
        p.half = h & 1;
    }
    int before = 0;
    for (int c = 0;;) {
        const uint64_t past = __ballot((before + sum) * tiles_n > want);
        if (past) {
            const int l = __builtin_ctzll(past);
            p.e = c + l;
            p.row_tiles = __builtin_amdgcn_readlane(t, l);
            p.tile = want - (before + __builtin_amdgcn_readlane(sum, l) - p.row_tiles) * tiles_n;
            return p.tile >= 0;
        }
        before += __builtin_amdgcn_readlane(sum, 63);
        if ((c += 64) >= n_groups)
            return false;
        t = lane_tiles<BM>(off, n_groups, c, rows, sum);
    }
}

// The epilogue's matrices from row lo on.
__device__ __forceinline__ void from_row(EpiArgs &args, int64_t lo)
{
    args.C = static_cast<char *>(args.C) + lo * args.ldc * (args.c_bf16 ? 2 : 4);
    if (args.residual)
        args.residual = static_cast<const char *>(args.residual) + lo * args.ldr * (args.r_bf16 ? 2 : 4);
    if (args.z)
        args.z = static_cast<char *>(args.z) + lo * args.ldz * 2;
}

constexpr int kRunM = 6;

// C[r] = epilogue(A[r] B_e) for the rows r of every group e.  The grid is the
// most blocks the row count allows; those past the real tiles leave.
template <int BM, int BN, bool B_KOUTER>
__global__ __launch_bounds__(kGT) void grouped_rows_kernel(const int64_t *__restrict__ off, int n_groups,
                                                           int64_t rows, int64_t N, int64_t K,
                                                           const uint16_t *__restrict__ A, int64_t lda,
                                                           const uint16_t *__restrict__ B, int64_t ldb,
                                                           int64_t stride_b, EpiArgs args, int tiles_n,
                                                           int cus)
{
    Place p;
    if (!find_tile<BM>(off, n_groups, rows, tiles_n, cus, p))
        return;
    // A group's row tiles walk its columns together, in equal runs of at most
    // kRunM, so that one fetch of a W column serves all of them.
    int tm, tn;
    const int e = p.e, runs = (p.row_tiles + kRunM - 1) / kRunM;
    grouped(p.tile, p.row_tiles, tiles_n, tm, tn, (p.row_tiles + runs - 1) / runs);
    int64_t lo, hi;
    group_range(off, e, rows, lo, hi);
    const int64_t M = hi - lo, n0 = (int64_t)tn * BN;
    const int64_t m0 = (int64_t)tm * BM + (p.half > 0 ? BM / 2 : 0);
    if (m0 >= M || n0 >= N)  // an empty half, or offsets that decrease
        return;
    const bool half = BM == kBM && (p.half >= 0 || M - m0 <= BM / 2);
    from_row(args, lo);
    A += lo * lda;
    B += e * stride_b;
    if constexpr (B_KOUTER && BM == kBM) {
        ZS_AP;
        if (half)
            gemm_tile_ap<kBM / 2>(M, N, K, A, lda, B, ldb, epi, m0, n0, (ZS_LDS char *)pa0, (ZS_LDS char *)pa1,
                                  Bs);
        else
            gemm_tile_ap<kBM>(M, N, K, A, lda, B, ldb, epi, m0, n0, (ZS_LDS char *)pa0, (ZS_LDS char *)pa1, Bs);
    } else if constexpr (B_KOUTER) {
        ZS_STAGES(BM, BN);
        const LayerEpi epi{args, ZS_CORNER};
        gemm_tile<BM, BN, false, true>(M, N, K, A, lda, B, ldb, epi, m0, n0, As, Bs);
    } else {
        ZS_PAIRS(BM, BN);
        const LayerEpi epi{args, ZS_CORNER_KP((BM < BN ? BM : BN) * 64)};
        if (half)
            gemm_tile_kp<kBM / 2, BN>(M, N, K, A, lda, B, ldb, epi, m0, n0, ZS_P);
        else
            gemm_tile_kp<BM, BN>(M, N, K, A, lda, B, ldb, epi, m0, n0, ZS_P);
    }
}

// The same with few rows in all, in 32-row tiles.
template <int BN, bool B_KOUTER>
__global__ __launch_bounds__(kGT) void grouped_skinny_kernel(const int64_t *__restrict__ off, int n_groups,
                                                             int64_t rows, int64_t N, int64_t K,
                                                             const uint16_t *__restrict__ A, int64_t lda,
                                                             const uint16_t *__restrict__ B, int64_t ldb,
                                                             int64_t stride_b, EpiArgs args, int tiles_n,
                                                             int cus)
{
    Place p;
    if (!find_tile<kSkM>(off, n_groups, rows, tiles_n, cus, p))
        return;
    const int64_t m0 = (int64_t)(p.tile % p.row_tiles) * kSkM, n0 = (int64_t)(p.tile / p.row_tiles) * BN;
    int64_t lo, hi;
    group_range(off, p.e, rows, lo, hi);
    const int64_t M = hi - lo;
    if (m0 >= M || n0 >= N)
        return;
    from_row(args, lo);
    A += lo * lda;
    B += p.e * stride_b;
    if constexpr (BN == kOuN)
        skinny_outer_tile(M, N, K, A, lda, B, ldb, args, m0, n0);
    else
        skinny_tile<B_KOUTER>(M, N, K, A, lda, B, ldb, args, m0, n0);
}

// How a weight gradient is stored.  fp32 in whole 128-byte lines goes past the
// caches (nontemporal: 4 to 20 % on 64 groups, 2048 x 1408); rows that begin inside
// a line do not, as their lines come in two parts that only a cache puts
// together: 25 groups of 7 rows, 2136 x 7224, 320 us against 680, of 240 rows 522 and
// 825; 4096 x 14344 from 4096 tokens in 8 bits 432 and 454.
constexpr int kOutFp32 = 0, kOutBf16 = 1, kOutLines = 2;

// C_e = sum over the rows r of group e of A[r]^T B[r]; an empty group's C_e is
// zeros.
template <int BM, int BN, int OUT>
__global__ __launch_bounds__(kGT, BM == BN ? 2 : 4)
void grouped_depth_kernel(const int64_t *__restrict__ off, int64_t rows, int64_t M, int64_t N,
                          const uint16_t *__restrict__ A, int64_t lda, const uint16_t *__restrict__ B,
                          int64_t ldb, void *__restrict__ C, int64_t ldc, int64_t stride_c, int tiles_m,
                          int tiles_n)
{
    constexpr int ST = BM == BN ? 4 : 3;
    __shared__ __attribute__((aligned(1024))) char a0[BM * 64], a1[BM * 64], a2[BM * 64];
    __shared__ __attribute__((aligned(1024))) char b0[BN * 64], b1[BN * 64], b2[BN * 64];
    __shared__ __attribute__((aligned(1024))) char a3[ST > 3 ? BM * 64 : 16], b3[ST > 3 ? BN * 64 : 16];
    ZS_LDS char *As[ST], *Bs[ST];
    As[0] = (ZS_LDS char *)a0, As[1] = (ZS_LDS char *)a1, As[2] = (ZS_LDS char *)a2;
    Bs[0] = (ZS_LDS char *)b0, Bs[1] = (ZS_LDS char *)b1, Bs[2] = (ZS_LDS char *)b2;
    if constexpr (ST > 3)
        As[ST - 1] = (ZS_LDS char *)a3, Bs[ST - 1] = (ZS_LDS char *)b3;
    const int per = tiles_m * tiles_n;
    const int i = xcd_order(blockIdx.x, gridDim.x);
    const int e = i / per;
    // Along C's rows, so that what is stored together lies together: 25 groups of
    // 7 rows, 2048 x 7168: 271 us against 287 in blocks of eight row tiles.
    const int tm = (i - e * per) / tiles_n, tn = (i - e * per) % tiles_n;
    int64_t lo, hi;
    group_range(off, e, rows, lo, hi);
    const PlainEpi<OUT == kOutBf16, OUT == kOutLines> epi{
        static_cast<char *>(C) + e * stride_c * (OUT == kOutBf16 ? 2 : 4), ldc};
    gemm_tile<BM, BN, true, true>(M, N, hi - lo, A + lo * lda, lda, B + lo * ldb, ldb, epi,
                                  (int64_t)tm * BM, (int64_t)tn * BN, As, Bs);
}

// ------------------------------------------- products from 8-bit operands --

// C = A^T B with A a K x M checkpoint (codes and exponent bytes) and B bf16,
// both K-outer.  The pipeline is gemm_tile's; what differs is A.
//
// A stage holds 32 k rows of BM code bytes.  The blocks run along k, so one
// row of exponent bytes serves a stage and a lane, which holds one row of C,
// needs one exponent a stage.  A fragment is one ds_read_b64_tr_b8 (an 8 x 16
// byte block transposed over 16 lanes: eight k of one row) and four
// v_cvt_scalef32_pk_bf16_fp8, exact.  The 8 waves stand 4 x 2, each (BM / 4) x
// (BN / 2): that halves the conversions of gemm_tile's 2 x 4 (each A fragment
// is then widened by two waves instead of four) for the same accumulators.
//
// The 32-byte unit U of k row kr sits at U ^ (kr & 7) (BM = 256; for BM = 128,
// whose rows are half as long, U ^ ((kr >> 1) & 3)), so that the eight k rows
// a half wave reads at once fall into eight different bank ranges.
//
// Exponents travel four tiles at a time, one 256-byte row a wave (waves 4-7
// repeat 0-3): fetched in the first tile of a group behind its barrier, when
// every wave has the present group's bytes in registers, read in the last.
// A wave's wait counts its own instructions back from the newest; the extra
// one makes it stricter, never laxer.
template <int BM>
__device__ __forceinline__ int a8_swz(int kr) { return BM == 256 ? kr & 7 : (kr >> 1) & 3; }

template <int BM, int BN, class Epi>
__device__ __forceinline__ void gemm_tile_a8(int64_t M, int64_t N, int64_t K,
                                             const uint8_t *__restrict__ A, int64_t lda,
                                             const uint8_t *__restrict__ E, int64_t lde,
                                             const uint16_t *__restrict__ B, int64_t ldb, const Epi &epi,
                                             int64_t m0, int64_t n0, ZS_LDS char *const (&As)[kStages],
                                             ZS_LDS char *Es, ZS_LDS char *const (&Bs)[kStages])
{
    static_assert(BM == 256 || BM == 128, "");
    constexpr int TM = BM / 128, TN = BN / 64;
    constexpr int NMF = TM * TN, NRD = TM + 2 * TN, NQ = NMF < NRD ? NMF : NRD;
    constexpr int NIB = Op<BN, true>::NI;
    constexpr int D = 1 + NIB;

    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = (wave >> 1) * (BM / 4), wn = (wave & 1) * (BN / 2);
    const int fr = lane & 31, fh = lane >> 5;

    // A's 1 KB instruction I: k rows KPI I .. of BM bytes.  A stage of 128
    // rows is four of them; waves 4-7 repeat what waves 0-3 fetch.
    constexpr int KPI = 1024 / BM, LPR = BM / 16;
    const int I = BM == 256 ? wave : wave & 3;
    uint32_t va, vb[2];
    {
        const int kr = KPI * I + lane / LPR, slot = lane % LPR;
        const int c16 = (((slot >> 1) ^ a8_swz<BM>(kr)) << 1) | (slot & 1);
        va = (uint32_t)(kr * lda + 16 * c16);
    }
#pragma unroll
    for (int n = 0; n < 2; ++n)
        vb[n] = n < NIB ? dma_offset<BN, true>(ldb, wave, lane, n) : 0u;
    int fa_off[TM][2], fb_off[TN][2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int j = lane & 15, kr = 16 * s + 8 * fh + (j >> 1);
#pragma unroll
        for (int i = 0; i < TM; ++i)
            fa_off[i][s] = kr * BM + ((((wm + 32 * i) >> 5) ^ a8_swz<BM>(kr)) << 5) +
                           16 * ((lane >> 4) & 1) + 8 * (j & 1);
#pragma unroll
        for (int j2 = 0; j2 < TN; ++j2)
            fb_off[j2][s] = frag_offset<BN, true>(wn + 32 * j2, s, lane);
    }
    const int fe_off = wm + fr;

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v)
                acc[i][j][v] = 0.0f;

    const int64_t kt_n = (K + kBK - 1) / kBK;
    auto dma = [&](auto st, int64_t kt) {
        constexpr int S = decltype(st)::value;
        const int64_t k0 = kt * kBK;
        const __amdgpu_buffer_rsrc_t ra = rsrc(A + k0 * lda + m0, (K - 1 - k0) * lda + M - m0);
        const __amdgpu_buffer_rsrc_t rb = rsrc(B + k0 * ldb + n0, ((K - 1 - k0) * ldb + N - n0) * 2);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (ZS_LDS void *)(As[S] + I * 1024), 16, va, 0, 0, 0);
#pragma unroll
        for (int n = 0; n < NIB; ++n)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (ZS_LDS void *)(Bs[S] + (wave + kNW * n) * 1024),
                                                     16, vb[n], 0, 0, 0);
    };
    // Exponent rows kt .. kt + 3 (past the last: the last again).
    auto dma_exps = [&](int64_t kt) {
        const int64_t r = kt + (wave & 3) < kt_n ? kt + (wave & 3) : kt_n - 1;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc(E + r * lde + m0, M - m0),
                                                 (ZS_LDS void *)(Es + (wave & 3) * 256), 4, 4 * lane, 0, 0,
                                                 0);
    };
    typedef int i32x2 __attribute__((ext_vector_type(2)));
    i32x2 ra0[TM], ra1[TM];
    bf16x8 fb0[TN], fb1[TN];
    uint32_t ex[kStages][TM];
    auto frags = [&](auto st, int s, i32x2 (&fa)[TM], bf16x8 (&fb)[TN]) {
        constexpr int S = decltype(st)::value;
#pragma unroll
        for (int i = 0; i < TM; ++i)
            fa[i] = __builtin_amdgcn_ds_read_tr8_b64_v2i32((ZS_LDS i32x2 *)(As[S] + fa_off[i][s]));
#pragma unroll
        for (int j = 0; j < TN; ++j)
            fb[j] = frag_read<BN, true>(Bs[S], fb_off[j][s]);
    };
    auto exps = [&]() {
#pragma unroll
        for (int r = 0; r < kStages; ++r)
#pragma unroll
            for (int i = 0; i < TM; ++i)
                ex[r][i] = *reinterpret_cast<const ZS_LDS uint8_t *>(Es + 256 * r + fe_off + 32 * i);
    };
    auto widen = [&](i32x2 w, uint32_t byte) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        const float s = __uint_as_float(byte << 23);
        const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)w[0], s, false);
        const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)w[0], s, true);
        const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)w[1], s, false);
        const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)w[1], s, true);
        return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    };
    auto mma = [&](const bf16x8 (&fa)[TM], const bf16x8 (&fb)[TN], int lo, int hi) {
#pragma unroll
        for (int q = 0; q < NMF; ++q)
            if (q >= lo && q < hi)
                acc[q / TN][q % TN] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                    fa[q / TN], fb[q % TN], acc[q / TN][q % TN], 0, 0, 0);
    };
    auto wait_for = [&](int64_t kt1) {
        const int64_t after = kt_n - 1 - kt1;
        if (after >= 2)
            wait_vm_lgkm0<2 * D>();
        else if (after == 1)
            wait_vm_lgkm0<D>();
        else
            wait_vm_lgkm0<0>();
    };
    // Tile kt in stage S, the S-th of its group of four, as in gemm_tile.
    auto tile = [&](auto st, auto steady, int64_t kt) {
        constexpr int S = decltype(st)::value;
        constexpr bool STEADY = decltype(steady)::value != 0;
        constexpr int SN = (S + kStages - 1) % kStages, S1 = (S + 1) % kStages;
        __builtin_amdgcn_sched_barrier(0);
        bf16x8 fa[TM], fc[TM];
        if (STEADY || kt + kStages - 1 < kt_n)
            dma(IC<SN>{}, kt + kStages - 1);
        frags(IC<S>{}, 1, ra1, fb1);
#pragma unroll
        for (int i = 0; i < TM; ++i)
            fa[i] = widen(ra0[i], ex[S][i]);
        mma(fa, fb0, 0, NMF);
        seq<NQ, NMF, NRD, STEADY ? D : 0>();
#pragma unroll
        for (int i = 0; i < TM; ++i)
            fc[i] = widen(ra1[i], ex[S][i]);
        mma(fc, fb1, 0, NMF / 2);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (STEADY)
            wait_vm_lgkm0<2 * D>();
        else
            wait_for(kt + 1);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        if (S == 0 && (STEADY || kt + kStages < kt_n))
            dma_exps(kt + kStages);
        if (STEADY || kt + 1 < kt_n) {
            frags(IC<S1>{}, 0, ra0, fb0);
            if (S == kStages - 1)
                exps();
        }
        mma(fc, fb1, NMF / 2, NMF);
        seq<NQ, NMF - NMF / 2, NRD, 0>();
    };
    if (kt_n > 0) {
        dma_exps(0);
        dma(IC<0>{}, 0);
        if (kt_n > 1)
            dma(IC<1>{}, 1);
        if (kt_n > 2)
            dma(IC<2>{}, 2);
        wait_for(0);
        __builtin_amdgcn_s_barrier();
        frags(IC<0>{}, 0, ra0, fb0);
        exps();
        int64_t kt = 0;
        // groups whose tiles kt + 3 .. kt + 6 exist
        for (; kt + 2 * kStages - 1 <= kt_n; kt += kStages) {
            tile(IC<0>{}, IC<1>{}, kt);
            tile(IC<1>{}, IC<1>{}, kt + 1);
            tile(IC<2>{}, IC<1>{}, kt + 2);
            tile(IC<3>{}, IC<1>{}, kt + 3);
        }
        for (; kt < kt_n; kt += kStages) {
            tile(IC<0>{}, IC<0>{}, kt);
            if (kt + 1 < kt_n)
                tile(IC<1>{}, IC<0>{}, kt + 1);
            if (kt + 2 < kt_n)
                tile(IC<2>{}, IC<0>{}, kt + 2);
            if (kt + 3 < kt_n)
                tile(IC<3>{}, IC<0>{}, kt + 3);
        }
    }
    epi.template tile32<TM, TN>(acc, m0 + wm, n0 + wn, M, N, lane);
}

template <int BM, int BN, int OUT>
__global__ __launch_bounds__(kGT) void saved_kernel(int64_t M, int64_t N, int64_t K,
                                                    const uint8_t *__restrict__ A, int64_t lda,
                                                    const uint8_t *__restrict__ E, int64_t lde,
                                                    const uint16_t *__restrict__ B, int64_t ldb,
                                                    void *__restrict__ C, int64_t ldc, int tiles_m,
                                                    int tiles_n, int n_big)
{
    __shared__ __attribute__((aligned(1024))) char a0[BM * 32], a1[BM * 32], a2[BM * 32], a3[BM * 32];
    __shared__ __attribute__((aligned(1024))) char b0[BN * 64], b1[BN * 64], b2[BN * 64], b3[BN * 64];
    __shared__ __attribute__((aligned(256))) char es[1024];
    ZS_LDS char *const As[kStages] = {(ZS_LDS char *)a0, (ZS_LDS char *)a1, (ZS_LDS char *)a2,
                                      (ZS_LDS char *)a3};
    ZS_LDS char *const Bs[kStages] = {(ZS_LDS char *)b0, (ZS_LDS char *)b1, (ZS_LDS char *)b2,
                                      (ZS_LDS char *)b3};
    ZS_LDS char *const Es = (ZS_LDS char *)es;
    const PlainEpi<OUT == kOutBf16, OUT == kOutLines> epi{C, ldc};
    int64_t m0, n0;
    if (place<BM, BN>(tiles_m, tiles_n, n_big, m0, n0))
        gemm_tile_a8<BM, BN>(M, N, K, A, lda, E, lde, B, ldb, epi, m0, n0, As, Es, Bs);
    else if constexpr (BM == kBM)
        gemm_tile_a8<BM / 2, BN>(M, N, K, A, lda, E, lde, B, ldb, epi, m0, n0, As, Es, Bs);
}

}  // namespace

// The epilogue of an M x N product, checked and translated.  `offsets` (NULL: no
// groups) refuses what needs rows counted from a multiple of 32.
zero_status epilogue_check(int64_t M, int64_t N, const void *A, const void *B, const void *C, int64_t ldc,
                           int32_t c_dtype, const zero_epilogue *ep, const int64_t *offsets)
{
    if (M == 0 || N == 0)
        return ZERO_OK;
    const bool grouped = offsets != nullptr;
    if (is_one_of(C, {A, B, offsets}))
        return fail(ZERO_ERR_INVALID_ARG, "C must not be an operand");
    if (!ep)
        return ZERO_OK;
    if (ep->act < ZERO_ACT_NONE || ep->act > ZERO_ACT_SILU)
        return fail(ZERO_ERR_INVALID_ARG, "unknown activation %d", ep->act);
    zero_status st;
    if (ep->bias) {
        if (grouped)
            return fail(ZERO_ERR_UNSUPPORTED, "a grouped product takes no bias");
        if ((st = check_matrix("bias", ep->bias, N, N, ep->bias_dtype)) != ZERO_OK)
            return st;
        if (ep->bias == C)
            return fail(ZERO_ERR_INVALID_ARG, "bias must not lie where C is written");
    }
    if (ep->residual) {
        if ((st = check_matrix("residual", ep->residual, ep->ldr, N, ep->residual_dtype)) != ZERO_OK ||
            (st = check_extent(M, N, ep->ldr)) != ZERO_OK)
            return st;
        if (ep->residual == C && (ep->residual_dtype != c_dtype || ep->ldr != ldc))
            return fail(ZERO_ERR_INVALID_ARG, "a residual in place of C needs C's type and leading dimension");
    }
    // What is kept must not lie where the product still reads or writes.
    auto apart = [&](const zero_saved *s, const zero_saved *other) {
        for (const void *p : {data_of(s), scales_of(s)})
            if (is_one_of(p, {C, A, B, offsets, ep->residual, ep->bias, data_of(other), scales_of(other)}))
                return false;
        return data_of(s) != scales_of(s);
    };
    if (ep->preact) {
        if ((st = saved_check("preact", ep->preact, M, N)) != ZERO_OK)
            return st;
        if (!apart(ep->preact, ep->output))
            return fail(ZERO_ERR_INVALID_ARG, "preact needs a buffer of its own");
        if (grouped && ep->preact->format != ZERO_SAVED_BF16)
            return fail(ZERO_ERR_UNSUPPORTED, "a grouped product keeps its pre-activation in bf16 only");
    }
    if (ep->output) {
        if (grouped)
            return fail(ZERO_ERR_UNSUPPORTED, "a grouped product keeps no 8-bit output");
        if ((st = saved_check("output", ep->output, M, N)) != ZERO_OK)
            return st;
        if (ep->output->format != ZERO_SAVED_E4M3)
            return fail(ZERO_ERR_UNSUPPORTED, "output is kept in 8 bits only");
        if (!apart(ep->output, ep->preact))
            return fail(ZERO_ERR_INVALID_ARG, "output needs a buffer of its own");
    }
    return ZERO_OK;
}

namespace {

EpiArgs epi_args(const zero_epilogue *ep, void *C, int64_t ldc, int32_t c_dtype)
{
    EpiArgs a = {};
    a.C = C;
    a.ldc = ldc;
    a.c_bf16 = c_dtype == ZERO_BF16;
    a.vec = vec16(C, ldc, bytes_of(c_dtype));
    if (!ep)
        return a;
    a.act = ep->act;
    a.bias = ep->bias;
    a.bias_bf16 = ep->bias_dtype == ZERO_BF16;
    a.residual = ep->residual;
    a.ldr = ep->ldr;
    a.r_bf16 = ep->residual_dtype == ZERO_BF16;
    if (ep->residual)
        a.vec = a.vec && vec16(ep->residual, ep->ldr, bytes_of(ep->residual_dtype));
    if (ep->preact) {
        a.z = ep->preact->data;
        a.ldz = ep->preact->ld;
        if (ep->preact->format == ZERO_SAVED_E4M3) {
            a.z_scales = ep->preact->scales;
            a.ldzs = ep->preact->ld_scales;
        } else {
            a.vec = a.vec && vec16(a.z, a.ldz, 2);
        }
    }
    if (ep->output) {
        a.o = static_cast<uint8_t *>(ep->output->data);
        a.ldo = ep->output->ld;
        a.o_scales = ep->output->scales;
        a.ldos = ep->output->ld_scales;
    }
    return a;
}

constexpr int64_t kMaxBlocks = int64_t(0xffffffffu) / (2 * kGT);

}  // namespace

// zero_gemm_saved_bf16's checks, with nothing launched.
zero_status gemm_saved_check(int64_t M, int64_t N, int64_t K, const zero_saved *A, const uint16_t *B,
                             int64_t ldb, const void *C, int64_t ldc, int32_t c_dtype)
{
    if (M < 0 || N < 0 || K < 0)
        return fail(ZERO_ERR_INVALID_ARG, "negative GEMM size");
    if (!known_dtype(c_dtype))
        return fail(ZERO_ERR_INVALID_ARG, "unknown C dtype %d", c_dtype);
    if (M == 0 || N == 0)
        return ZERO_OK;
    zero_status st;
    if ((st = saved_check("A", A, K, M)) != ZERO_OK ||
        (st = check_matrix("B", operand(B, K > 0), ldb, N, ZERO_BF16)) != ZERO_OK ||
        (st = check_matrix("C", C, ldc, N, c_dtype)) != ZERO_OK)
        return st;
    if (is_one_of(C, {A->data, scales_of(A), B}))
        return fail(ZERO_ERR_INVALID_ARG, "C must not be an operand");
    if (M % 8 || N % 8 || ldb % 8 || A->ld % 8)
        return fail(ZERO_ERR_UNSUPPORTED, "a product from a kept operand needs M, N and the leading "
                    "dimensions multiples of 8");
    if (A->format == ZERO_SAVED_E4M3 && (A->ld_scales % 4 || !aligned(A->scales, 4)))
        return fail(ZERO_ERR_UNSUPPORTED, "the scales of a product's operand must be 4-byte aligned rows");
    if (A->ld > (int64_t(1) << 25) || ldb > (int64_t(1) << 25))
        return fail(ZERO_ERR_UNSUPPORTED, "leading dimension too large for 32-bit operand offsets (at most "
                    "%lld)", 1ll << 25);
    if (!aligned(A->data, 16) || !aligned(B, 16))
        return fail(ZERO_ERR_ALIGNMENT, "A and B must be 16-byte aligned");
    const int64_t tm = (M + kBM - 1) / kBM, tn = (N + kBN - 1) / kBN;
    if (tm > kMaxBlocks / tn)
        return fail(ZERO_ERR_UNSUPPORTED, "too many GEMM tiles for one launch");
    return ZERO_OK;
}

static int out_kind(const void *C, int64_t ldc, int64_t stride_c, int32_t c_dtype)
{
    if (c_dtype == ZERO_BF16)
        return kOutBf16;
    return aligned(C, 128) && ldc % 32 == 0 && stride_c % 32 == 0 ? kOutLines : kOutFp32;
}

zero_status gemm_saved_run(int64_t M, int64_t N, int64_t K, const zero_saved *A, const uint16_t *B,
                           int64_t ldb, void *C, int64_t ldc, int32_t c_dtype, hipStream_t s)
{
    if (M == 0 || N == 0)
        return ZERO_OK;
    if (A->format == ZERO_SAVED_BF16)
        return gemm_run(M, N, K, static_cast<const uint16_t *>(A->data), A->ld, ZERO_K_OUTER, B, ldb,
                        ZERO_K_OUTER, C, ldc, c_dtype, s);
    const uint8_t *codes = static_cast<const uint8_t *>(A->data);
    (void)hipGetLastError();
    const int out = out_kind(C, ldc, 0, c_dtype);
#define ZS_SAVED(BM_, BN_, OUT)                                                                    \
    hipLaunchKernelGGL((saved_kernel<BM_, BN_, OUT>), g.grid, dim3(kGT), 0, s, M, N, K, codes, A->ld, \
                       A->scales, A->ld_scales, B, ldb, C, ldc, g.tm, g.tn, g.n_big)
    if (small_tiles(M, N)) {
        const Grid g = tiles(M, N, 128, 128, false);
        if (out == kOutBf16)
            ZS_SAVED(128, 128, kOutBf16);
        else if (out == kOutLines)
            ZS_SAVED(128, 128, kOutLines);
        else
            ZS_SAVED(128, 128, kOutFp32);
    } else {
        const Grid g = tiles(M, N, kBM, kBN, true);
        if (out == kOutBf16)
            ZS_SAVED(kBM, kBN, kOutBf16);
        else if (out == kOutLines)
            ZS_SAVED(kBM, kBN, kOutLines);
        else
            ZS_SAVED(kBM, kBN, kOutFp32);
    }
#undef ZS_SAVED
    return launched("gemm_saved");
}

// Up to two blocks a CU of 32 x 32 tiles: 1 x 4096 x 14336 takes 55 us so
// (K-inner B 31) and 95 in 128 x 128 tiles, 128 x 4096 x 4096 22 and 32,
// 256 x 1024 x 1024 7.2 and 13; past that, with 64 x 14336 x 4096, 60 and
// 44, 512 x 4096 x 4096 80 and 34.  Of a K-outer B more than one block a CU
// becomes 32 x 64 tiles, up to one a CU (with two, 448 blocks, 64 x 14336 x 4096
// takes 48 us and 44 in 128 x 128 ones, 1 x 28672 x 8192 103 and 85); so do
// leading dimensions for which the 64 k rows of a 32-column stage would pass
// 32-bit offsets.
//
// Grouped products by the same rule, with the row tiles that the groups may
// have, against 128 x 128 tiles (K-outer and K-inner B): 2 groups of a row, 14336 ->
// 4096, 60 and 48 us against 124 and 207; 16 of one, 4096 -> 1024, 34 and 43
// against 46 and 65; 4 of 100, 2048 -> 512, 9.1 and 8.0 against 22 and 26.
//
// Columns of a few-row tile, 0 where the product takes larger ones.
static int skinny_columns(int64_t row_tiles, int64_t N, bool b_kouter, int64_t ldb)
{
    const int64_t sn = (N + kSkN - 1) / kSkN, cus = cu_count();
    if (row_tiles > 2 * cus / sn)
        return 0;
    return !b_kouter || (row_tiles * sn <= cus && ldb <= (int64_t(1) << 24)) ? kSkN : kOuN;
}

zero_status epilogue_gemm_run(int64_t M, int64_t N, int64_t K, const uint16_t *A, int64_t lda,
                              int32_t a_order, const uint16_t *B, int64_t ldb, int32_t b_order, void *C,
                              int64_t ldc, int32_t c_dtype, const zero_epilogue *ep, hipStream_t s)
{
    if (M == 0 || N == 0)
        return ZERO_OK;
    const EpiArgs a = epi_args(ep, C, ldc, c_dtype);
    const bool ao = a_order == ZERO_K_OUTER, bo = b_order == ZERO_K_OUTER;
    const bool small = small_tiles(M, N);
    // Under 1024 the halves' final exchange is not earned back: 1000 x 1000 x 600
    // with a K-inner B takes 15.3 us with it and 13.9 without.
    const bool k2 = small && K >= 1024;
    const Grid g = small ? tiles(M, N, 128, 128, false) : tiles(M, N, kBM, kBN, true);
    (void)hipGetLastError();
    if (const int bn = ao ? 0 : skinny_columns((M + kSkM - 1) / kSkM, N, bo, ldb)) {
        const int64_t sm = (M + kSkM - 1) / kSkM;
        const dim3 grid((unsigned)(sm * ((N + bn - 1) / bn)));
#define ZS_SKINNY(BN_, BO)                                                                         \
    hipLaunchKernelGGL((skinny_kernel<BN_, BO>), grid, dim3(kGT), 0, s, M, N, K, A, lda, B, ldb, a, (int)sm)
        if (!bo)
            ZS_SKINNY(kSkN, false);
        else if (bn == kSkN)
            ZS_SKINNY(kSkN, true);
        else
            ZS_SKINNY(kOuN, true);
#undef ZS_SKINNY
        return launched("gemm_epilogue");
    }
#define ZS_EPI(AO, BO)                                                                             \
    do {                                                                                           \
        if (k2)                                                                                    \
            hipLaunchKernelGGL((epi_kernel_k2<AO, BO>), g.grid, dim3(kGT), 0, s, M, N, K, A, lda,  \
                               B, ldb, a, g.tm, g.tn);                                             \
        else if (small)                                                                                 \
            hipLaunchKernelGGL((epi_kernel<128, 128, AO, BO>), g.grid, dim3(kGT), 0, s, M, N, K, A, \
                               lda, B, ldb, a, g.tm, g.tn, g.n_big);                               \
        else                                                                                       \
            hipLaunchKernelGGL((epi_kernel<kBM, kBN, AO, BO>), g.grid, dim3(kGT), 0, s, M, N, K, A, \
                               lda, B, ldb, a, g.tm, g.tn, g.n_big);                               \
    } while (0)
    if (ao && bo) {
        ZS_EPI(true, true);
    } else if (ao) {
        ZS_EPI(true, false);
    } else if (bo && !small) {
        hipLaunchKernelGGL(epi_kernel_ap, g.grid, dim3(kGT), 0, s, M, N, K, A, lda, B, ldb, a, g.tm, g.tn,
                           g.n_big);
    } else if (bo && k2) {
        hipLaunchKernelGGL((epi_kernel_k2<false, true>), g.grid, dim3(kGT), 0, s, M, N, K, A, lda, B, ldb, a,
                           g.tm, g.tn);
    } else if (bo) {
        hipLaunchKernelGGL((epi_kernel<128, 128, false, true>), g.grid, dim3(kGT), 0, s, M, N, K, A, lda, B,
                           ldb, a, g.tm, g.tn, g.n_big);
    } else if (k2) {
        hipLaunchKernelGGL((epi_kernel_k2<false, false>), g.grid, dim3(kGT), 0, s, M, N, K, A, lda, B, ldb,
                           a, g.tm, g.tn);
    } else if (small) {
        hipLaunchKernelGGL((epi_kernel_kp<128, 128>), g.grid, dim3(kGT), 0, s, M, N, K, A, lda, B, ldb, a,
                           g.tm, g.tn, g.n_big);
    } else {
        hipLaunchKernelGGL((epi_kernel_kp<kBM, kBN>), g.grid, dim3(kGT), 0, s, M, N, K, A, lda, B, ldb, a,
                           g.tm, g.tn, g.n_big);
    }
#undef ZS_EPI
    return launched("gemm_epilogue");
}

// ------------------------------------------------------ grouped products --

zero_status grouped_check(int32_t n_groups, const int64_t *offsets, int64_t rows)
{
    if (n_groups < 1 || rows < 0)
        return fail(ZERO_ERR_INVALID_ARG, "a grouped product needs at least one group and rows >= 0");
    if (!offsets)
        return fail(ZERO_ERR_INVALID_ARG, "offsets is required");
    if (!aligned(offsets, 8))
        return fail(ZERO_ERR_ALIGNMENT, "offsets must be 8-byte aligned");
    return ZERO_OK;
}

// The most tiles of bm rows that n_groups groups over `rows` rows can have.
static int64_t most_tiles(int32_t n_groups, int64_t rows, int bm)
{
    const int64_t g = rows < n_groups ? rows : n_groups;
    return (rows + g * (bm - 1)) / bm;
}

zero_status grouped_rows_check(int32_t n_groups, const int64_t *offsets, int64_t rows, int64_t N, int64_t K,
                               const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb,
                               int32_t b_order, int64_t stride_b, const void *C, int64_t ldc,
                               int32_t c_dtype, const zero_epilogue *ep)
{
    zero_status st;
    if ((st = grouped_check(n_groups, offsets, rows)) != ZERO_OK ||
        (st = gemm_check(rows, N, K, operand(A, K > 0), lda, ZERO_K_INNER, operand(B, K > 0), ldb, b_order, C,
                         ldc, c_dtype)) != ZERO_OK ||
        (st = epilogue_check(rows, N, A, B, C, ldc, c_dtype, ep, offsets)) != ZERO_OK)
        return st;
    if (rows == 0 || N == 0)
        return ZERO_OK;
    const int64_t extent = b_order == ZERO_K_OUTER ? (K > 0 ? (K - 1) * ldb + N : 0) : (N - 1) * ldb + K;
    if (n_groups > 1 && (stride_b < extent || stride_b % 8))
        return fail(ZERO_ERR_INVALID_ARG, "stride_b must be a multiple of 8 and at least %lld (got %lld)",
                    (long long)extent, (long long)stride_b);
    if (stride_b > kMaxElems / n_groups)
        return fail(ZERO_ERR_UNSUPPORTED, "the groups' operands are too large");
    if (most_tiles(n_groups, rows, 128) > kMaxBlocks / ((N + 127) / 128))
        return fail(ZERO_ERR_UNSUPPORTED, "too many tiles for one launch");
    return ZERO_OK;
}

zero_status grouped_rows_run(int32_t n_groups, const int64_t *offsets, int64_t rows, int64_t N, int64_t K,
                             const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb,
                             int32_t b_order, int64_t stride_b, void *C, int64_t ldc, int32_t c_dtype,
                             const zero_epilogue *ep, hipStream_t s)
{
    if (rows == 0 || N == 0)
        return ZERO_OK;
    const EpiArgs a = epi_args(ep, C, ldc, c_dtype);
    // 128 x 128 tiles where 256 x 256 ones would leave half the CUs idle, and
    // where groups are short and two blocks a CU hide what a tile's start and
    // end cost.  Measured, 256 against 128: dX of 64 groups of 128 rows, 1408 ->
    // 2048, 101 and 95 us, of 192 rows 116 and 131; forward (K-outer B, where
    // gemm_tile_ap keeps up longer) 64 groups of 64 rows, 2048 -> 1408, 88 and 83,
    // of 128 rows 97 and 103, but 32 of 64 at 4096 -> 4096 182 and 217.
    const int cus = cu_count();
    const bool bo = b_order == ZERO_K_OUTER;
    (void)hipGetLastError();
    const int64_t sm = most_tiles(n_groups, rows, kSkM);
    if (const int bn = skinny_columns(sm, N, bo, ldb)) {
        const int tn = (int)((N + bn - 1) / bn);
        const dim3 grid((unsigned)(sm * tn));
#define ZS_SKINNY(BN_, BO)                                                                         \
    hipLaunchKernelGGL((grouped_skinny_kernel<BN_, BO>), grid, dim3(kGT), 0, s, offsets, n_groups, rows, N, K, \
                       A, lda, B, ldb, stride_b, a, tn, cus)
        if (!bo)
            ZS_SKINNY(kSkN, false);
        else if (bn == kSkN)
            ZS_SKINNY(kSkN, true);
        else
            ZS_SKINNY(kOuN, true);
#undef ZS_SKINNY
        return launched("gemm_grouped_rows");
    }
    const int64_t mean = rows / n_groups;
    const bool few = 2 * most_tiles(n_groups, rows, kBM) * ((N + kBN - 1) / kBN) <= cu_count();
    const bool small = few || (b_order == ZERO_K_INNER ? mean <= 128 : mean <= 64 && K <= 2048);
    const int bm = small ? 128 : kBM, bn = small ? 128 : kBN;
    const int tn = (int)((N + bn - 1) / bn);
    const dim3 grid((unsigned)(most_tiles(n_groups, rows, bm) * tn + (small ? 0 : cus / 2)));
#define ZS_ROWS(BM_, BN_, BO)                                                                      \
    hipLaunchKernelGGL((grouped_rows_kernel<BM_, BN_, BO>), grid, dim3(kGT), 0, s, offsets, n_groups, \
                       rows, N, K, A, lda, B, ldb, stride_b, a, tn, cus)
    if (b_order == ZERO_K_OUTER) {
        if (small)
            ZS_ROWS(128, 128, true);
        else
            ZS_ROWS(kBM, kBN, true);
    } else {
        if (small)
            ZS_ROWS(128, 128, false);
        else
            ZS_ROWS(kBM, kBN, false);
    }
#undef ZS_ROWS
    return launched("gemm_grouped_rows");
}

zero_status grouped_depth_check(int32_t n_groups, const int64_t *offsets, int64_t rows, int64_t M, int64_t N,
                                const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb,
                                const void *C, int64_t ldc, int64_t stride_c, int32_t c_dtype)
{
    zero_status st;
    // K rounded down to gemm_check's multiple of 8: with both operands
    // K-outer any number of rows will do.
    if ((st = grouped_check(n_groups, offsets, rows)) != ZERO_OK ||
        (st = gemm_check(M, N, rows / 8 * 8, operand(A, rows > 0), lda, ZERO_K_OUTER, operand(B, rows > 0),
                         ldb, ZERO_K_OUTER, C, ldc, c_dtype)) != ZERO_OK)
        return st;
    if (M == 0 || N == 0)
        return ZERO_OK;
    if (is_one_of(C, {A, B, offsets}))
        return fail(ZERO_ERR_INVALID_ARG, "C must not be an operand");
    if (n_groups > 1 && stride_c < (M - 1) * ldc + N)
        return fail(ZERO_ERR_INVALID_ARG, "stride_c must be at least %lld (got %lld)",
                    (long long)((M - 1) * ldc + N), (long long)stride_c);
    if (stride_c > kMaxElems / n_groups)
        return fail(ZERO_ERR_UNSUPPORTED, "the groups' results are too large");
    const int64_t per = ((M + 127) / 128) * ((N + 127) / 128);
    if (per > kMaxBlocks / n_groups)
        return fail(ZERO_ERR_UNSUPPORTED, "too many tiles for one launch");
    return ZERO_OK;
}

zero_status grouped_depth_run(int32_t n_groups, const int64_t *offsets, int64_t rows, int64_t M, int64_t N,
                              const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb, void *C,
                              int64_t ldc, int64_t stride_c, int32_t c_dtype, hipStream_t s)
{
    if (M == 0 || N == 0)
        return ZERO_OK;
    // Two 256 x 128 blocks a CU, three stages each, where the sums are so short
    // (128 rows a group on average) that a block is mostly its stores: 64 groups
    // of 64 rows, 2048 x 1408: 143 us against 160 with 256 x 256 tiles; of 256
    // rows 251 against 238, 8 of 512, 4096 x 14336, 707 against 670.  Likewise
    // where 256 x 256 tiles would leave half the CUs idle (4 groups of 300
    // rows, 512 x 512: 11.7 against 16.2 us).
    const int64_t wide = n_groups * ((M + kBM - 1) / kBM) * ((N + kBN - 1) / kBN);
    const bool narrow = rows / n_groups <= 128 || 2 * wide <= cu_count();
    const int bn = narrow ? kBN / 2 : kBN;
    const int tm = (int)((M + kBM - 1) / kBM), tn = (int)((N + bn - 1) / bn);
    const dim3 grid((unsigned)((int64_t)n_groups * tm * tn));
    (void)hipGetLastError();
    const int out = out_kind(C, ldc, stride_c, c_dtype);
#define ZS_DEPTH(BN_, OUT)                                                                         \
    hipLaunchKernelGGL((grouped_depth_kernel<kBM, BN_, OUT>), grid, dim3(kGT), 0, s, offsets, rows, M, N, \
                       A, lda, B, ldb, C, ldc, stride_c, tm, tn)
    if (out == kOutBf16) {
        if (narrow)
            ZS_DEPTH(kBN / 2, kOutBf16);
        else
            ZS_DEPTH(kBN, kOutBf16);
    } else if (out == kOutLines) {
        if (narrow)
            ZS_DEPTH(kBN / 2, kOutLines);
        else
            ZS_DEPTH(kBN, kOutLines);
    } else {
        if (narrow)
            ZS_DEPTH(kBN / 2, kOutFp32);
        else
            ZS_DEPTH(kBN, kOutFp32);
    }
#undef ZS_DEPTH
    return launched("gemm_grouped_depth");
}

}  // namespace zs

extern "C" {

zero_status zero_gemm_bf16_epilogue(int64_t M, int64_t N, int64_t K, const uint16_t *A, int64_t lda,
                                    int32_t a_order, const uint16_t *B, int64_t ldb, int32_t b_order,
                                    void *C, int64_t ldc, int32_t c_dtype, const zero_epilogue *epilogue,
                                    void *stream)
{
    zero_status st;
    if ((st = zs::gemm_check(M, N, K, zs::operand(A, K > 0), lda, a_order, zs::operand(B, K > 0), ldb, b_order,
                             C, ldc, c_dtype)) != ZERO_OK ||
        (st = zs::epilogue_check(M, N, A, B, C, ldc, c_dtype, epilogue, nullptr)) != ZERO_OK)
        return st;
    return zs::epilogue_gemm_run(M, N, K, A, lda, a_order, B, ldb, b_order, C, ldc, c_dtype, epilogue,
                                 static_cast<hipStream_t>(stream));
}

zero_status zero_gemm_saved_bf16(int64_t M, int64_t N, int64_t K, const zero_saved *A, const uint16_t *B,
                                 int64_t ldb, void *C, int64_t ldc, int32_t c_dtype, void *stream)
{
    const zero_status st = zs::gemm_saved_check(M, N, K, A, B, ldb, C, ldc, c_dtype);
    if (st != ZERO_OK)
        return st;
    return zs::gemm_saved_run(M, N, K, A, B, ldb, C, ldc, c_dtype, static_cast<hipStream_t>(stream));
}

zero_status zero_gemm_grouped_rows_bf16(int32_t n_groups, const int64_t *offsets, int64_t rows, int64_t N,
                                        int64_t K, const uint16_t *A, int64_t lda, const uint16_t *B,
                                        int64_t ldb, int32_t b_order, int64_t stride_b, void *C,
                                        int64_t ldc, int32_t c_dtype, const zero_epilogue *epilogue,
                                        void *stream)
{
    const zero_status st = zs::grouped_rows_check(n_groups, offsets, rows, N, K, A, lda, B, ldb, b_order,
                                                  stride_b, C, ldc, c_dtype, epilogue);
    if (st != ZERO_OK)
        return st;
    return zs::grouped_rows_run(n_groups, offsets, rows, N, K, A, lda, B, ldb, b_order, stride_b, C, ldc,
                                c_dtype, epilogue, static_cast<hipStream_t>(stream));
}

zero_status zero_gemm_grouped_depth_bf16(int32_t n_groups, const int64_t *offsets, int64_t rows, int64_t M,
                                         int64_t N, const uint16_t *A, int64_t lda, const uint16_t *B,
                                         int64_t ldb, void *C, int64_t ldc, int64_t stride_c,
                                         int32_t c_dtype, void *stream)
{
    const zero_status st = zs::grouped_depth_check(n_groups, offsets, rows, M, N, A, lda, B, ldb, C, ldc,
                                                   stride_c, c_dtype);
    if (st != ZERO_OK)
        return st;
    return zs::grouped_depth_run(n_groups, offsets, rows, M, N, A, lda, B, ldb, C, ldc, stride_c, c_dtype,
                                 static_cast<hipStream_t>(stream));
}

}  // extern "C"
