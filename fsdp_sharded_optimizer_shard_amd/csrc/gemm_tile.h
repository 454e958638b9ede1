// Tiles of the bf16 products: operand staging, the K loop and the plain
// epilogue, shared by the kernels of gemm.hip and layer.hip.  gemm.hip's head
// describes the tiling, the LDS layouts and the pipeline.
//
// A tile function ends by handing its accumulators to an epilogue object,
//   epi.tile32(acc, row0, col0, M, N, lane)   32 x 32 MFMA tiles, or
//   epi.tile16(acc, row0, col0, M, N, lane)   16 x 16 MFMA tiles,
// row0 and col0 being the wave's corner in C.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "internal.h"

namespace zs {
namespace {

constexpr int kNW = 8;          // waves per GEMM block: two per SIMD
constexpr int kGT = 64 * kNW;   // threads per GEMM block
constexpr int kBM = 256, kBN = 256, kBK = 32;
constexpr int kStages = 4;                 // LDS stages of kBK
constexpr int kStage = kBM * kBK * 2;      // bytes of one operand's stage
constexpr uint32_t kOOB = 0x80000000u;     // a buffer offset past every range
// Tile rows walked together.  Paired runs of the Mistral-7B MLP layer's
// GEMMs (distinct operands per launch): 4 rows beat 8 by 9 % on the dW
// products and 1-2 % on the others; 2, 6 and 16 were slower than 4.
constexpr int kGroupM = 4;

#define ZS_LDS __attribute__((address_space(3)))
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
template <int V>
using IC = std::integral_constant<int, V>;

__device__ __forceinline__ uint32_t f32_to_bf16_rne(float f)
{
    uint32_t u = __float_as_uint(f);
    if ((u & 0x7fffffffu) > 0x7f800000u)
        return 0x7fc0u;
    return (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
}

// K-inner stage of the 32x32x16 tile: byte offset of the 16-byte chunk c
// (of 4) of row r, swizzled by (r >> 2) & 3 so that the fragment reads are
// free of bank conflicts.
__device__ __forceinline__ int ki_swz(int r) { return (r >> 2) & 3; }
__device__ __forceinline__ int ki_pos(int r, int c) { return r * 64 + ((c ^ ki_swz(r)) << 4); }

// Buffer descriptor over `bytes` bytes from `base` (clamped to 2^31 - 1;
// the host bounds every offset below that).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void *base, int64_t bytes)
{
    int64_t n = bytes < 0 ? 0 : bytes;
    n = n > 0x7fffffffLL ? 0x7fffffffLL : n;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)n, 0x00020000);
}

// s_waitcnt vmcnt(V) lgkmcnt(0) (expcnt not waited).
template <int V>
__device__ __forceinline__ void wait_vm_lgkm0()
{
    static_assert(V >= 0 && V < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((V & 15) | ((V >> 4) << 14) | (0x7 << 4));
}

// A scheduling sequence of NQ groups sharing out NM MFMAs, NR LDS reads and
// NV global loads in order.
template <int NQ, int NM, int NR, int NV, int Q = 0>
__device__ __forceinline__ void seq()
{
    if constexpr (Q < NQ) {
        constexpr int m = NM * (Q + 1) / NQ - NM * Q / NQ;
        constexpr int r = NR * (Q + 1) / NQ - NR * Q / NQ;
        constexpr int v = NV * (Q + 1) / NQ - NV * Q / NQ;
        if constexpr (m > 0)
            __builtin_amdgcn_sched_group_barrier(0x008, m, 0);
        if constexpr (r > 0)
            __builtin_amdgcn_sched_group_barrier(0x100, r, 0);
        if constexpr (v > 0)
            __builtin_amdgcn_sched_group_barrier(0x020, v, 0);
        seq<NQ, NM, NR, NV, Q + 1>();
    }
}

// One operand's R x 32 stage.  Each of the 8 waves issues R / 128 DMA
// instructions of 1 KB; instruction n of wave w fills stage bytes
// [1024 I, 1024 I + 1024), I = w + 8 n, lane l landing at 16 l.
//   K-inner (rows of 64 B): rows 16 I .. +15; lane l takes row 16 I + l / 4
//     and stage slot l % 4, which holds k chunk slot ^ ((row >> 2) & 3).
//   K-outer (k-major, 2R bytes per k row): KPI = 1024 / 2R k rows per
//     instruction; lane l takes k row KPI I + l / (64 / KPI) and 16 bytes of
//     it.  The 32-byte unit of rows 16 u .. 16 u + 15 in k row kr sits at
//     unit_pos(u, kr) = u ^ (kr & 3) ^ ((u & 1) << 2): the transposing reads
//     of two neighbouring 16-row units then fall in different 128-byte
//     halves of the banks (2-way conflicts without the last term).
template <int R, bool KOUTER>
struct Op {
    static constexpr int NI = R / (16 * kNW);          // DMA instructions per wave per stage
    static constexpr int KPI = 1024 / (2 * R);         // K-outer: k rows per instruction
    static constexpr int NRD = KOUTER ? 2 : 1;         // LDS reads per fragment
};

__device__ __forceinline__ int unit_pos(int u, int kr) { return u ^ (kr & 3) ^ ((u & 1) << 2); }
// Inverse of unit_pos for one k row.
__device__ __forceinline__ int unit_at(int pos, int kr)
{
    const int x = pos ^ (kr & 3);
    return x ^ ((x & 1) << 2);
}

template <int R, bool KOUTER>
__device__ __forceinline__ uint32_t dma_offset(int64_t ld, int wave, int lane, int n)
{
    const int I = wave + kNW * n;
    if (!KOUTER) {
        const int r = 16 * I + (lane >> 2), c = (lane & 3) ^ ki_swz(r);
        return (uint32_t)((r * ld + 8 * c) * 2);
    }
    constexpr int KPI = Op<R, true>::KPI, LPR = 64 / KPI;  // lanes per k row
    const int kr = KPI * I + lane / LPR, w = (lane % LPR) * 16;
    const int lu = unit_at(w >> 5, kr), half = (w >> 4) & 1;
    return (uint32_t)((kr * ld + lu * 16 + half * 8) * 2);
}

// The k offset within the stage of a K-inner lane's chunk (for the K tail).
__device__ __forceinline__ int dma_kofs(int wave, int lane, int n)
{
    const int r = 16 * (wave + kNW * n) + (lane >> 2);
    return 8 * ((lane & 3) ^ ki_swz(r));
}

// First LDS read offset of the fragment of rows w0 .. w0 + 31 at k
// 16 s + 8 fh .. +7 (fh = lane / 32).  K-inner: one ds_read_b128.
// K-outer: two ds_read_b64_tr_b16, the second 4 k rows further; within
// 16-lane group g (lanes 16 g .. of each half-wave), lane j reads 8 bytes of
// k row 16 s + 8 fh + j / 4 at row offset 4 (j % 4) of unit (w0 + 16 g) / 16,
// and the transpose hands each lane the four k values of one row.
template <int R, bool KOUTER>
__device__ __forceinline__ int frag_offset(int w0, int s, int lane)
{
    const int fr = lane & 31, fh = lane >> 5;
    if (!KOUTER)
        return ki_pos(w0 + fr, 2 * s + fh);
    const int g = (lane >> 4) & 1, j = lane & 15, m = j >> 2, q = j & 3;
    const int kr = 16 * s + 8 * fh + m;  // the second read's k row kr + 4 has the same unit_pos
    return kr * (2 * R) + unit_pos((w0 + 16 * g) >> 4, kr) * 32 + q * 8;
}

template <int R, bool KOUTER>
__device__ __forceinline__ bf16x8 frag_read(const ZS_LDS char *stage, int off)
{
    if (!KOUTER)
        return *reinterpret_cast<const ZS_LDS bf16x8 *>(stage + off);
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZS_LDS s16x4 *)(stage + off));
    const s16x4 hi =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZS_LDS s16x4 *)(stage + off + 4 * (2 * R)));
    const s16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    return __builtin_bit_cast(bf16x8, v);
}

// XCD-contiguous order over a range of `n` blocks: block i of the range runs
// on XCD (first + i) % 8, and each XCD gets a contiguous run of the range.
__device__ __forceinline__ int xcd_order(int i, int n)
{
    const int per = n / 8, rem = n % 8, x = i % 8;
    return x * per + (x < rem ? x : rem) + i / 8;
}

// Grouped order: big tile `logical` -> (tile row, tile column), `group` tile
// rows at a time.
__device__ __forceinline__ void grouped(int logical, int tiles_m, int tiles_n, int &tm, int &tn,
                                        int group = kGroupM)
{
    const int gsz = group * tiles_n;
    const int g = logical / gsz;
    const int first_m = g * group;
    const int gm = tiles_m - first_m < group ? tiles_m - first_m : group;
    const int in_g = logical - g * gsz;
    tm = first_m + in_g % gm;
    tn = in_g / gm;
}

// The plain epilogue: C in fp32, or rounded to bf16.  STREAM stores fp32 past
// the caches, for results that nothing reads soon: dW of 64 experts of 256 rows
// (738 MB) 247 -> 238 us, of 8, 4096 x 14336 (1.9 GB), 571 -> 459.  Each store of a
// wave covers whole 128-byte lines.
template <bool OUT_BF16, bool STREAM = false>
struct PlainEpi {
    void *C;
    int64_t ldc;
    __device__ __forceinline__ void put(int64_t row, int64_t col, int64_t M, int64_t N, float x) const
    {
        if (row < M && col < N) {
            if (OUT_BF16)
                static_cast<uint16_t *>(C)[row * ldc + col] = (uint16_t)f32_to_bf16_rne(x);
            else if (STREAM)
                __builtin_nontemporal_store(x, static_cast<float *>(C) + row * ldc + col);
            else
                static_cast<float *>(C)[row * ldc + col] = x;
        }
    }
    template <int TM, int TN>
    __device__ __forceinline__ void tile32(const f32x16 (&acc)[TM][TN], int64_t row0, int64_t col0,
                                           int64_t M, int64_t N, int lane) const
    {
        const int fr = lane & 31, fh = lane >> 5;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    put(row0 + 32 * i + 8 * (v >> 2) + 4 * fh + (v & 3), col0 + 32 * j + fr, M, N,
                        acc[i][j][v]);
    }
    template <int TM, int TN>
    __device__ __forceinline__ void tile16(const f32x4 (&acc)[TM][TN], int64_t row0, int64_t col0,
                                           int64_t M, int64_t N, int lane) const
    {
        const int r16 = lane & 15, g = lane >> 4;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    put(row0 + 16 * i + 4 * g + v, col0 + 16 * j + r16, M, N, acc[i][j][v]);
    }
};

// One BM x BN tile of C (256 x 256, or 128 rows for half tiles, or
// 128 x 128): 8 waves in a 2 x 4 grid, each (BM / 2) x (BN / 4) as
// (BM / 64) x (BN / 128) MFMA tiles, over K stages of 32 (two substeps of
// 16).  Tile kt lives in LDS stage kt % ST; its DMA went out at the start of
// tile kt - ST + 1, so ST - 1 tiles of loads are in flight and no register
// staging or LDS write instruction is involved.
template <int BM, int BN, bool A_KOUTER, bool B_KOUTER, class Epi, int ST>
__device__ __forceinline__ void gemm_tile(int64_t M, int64_t N, int64_t K,
                                          const uint16_t *__restrict__ A, int64_t lda,
                                          const uint16_t *__restrict__ B, int64_t ldb,
                                          const Epi &epi, int64_t m0, int64_t n0,
                                          ZS_LDS char *const (&As)[ST],
                                          ZS_LDS char *const (&Bs)[ST])
{
    static_assert(ST == 3 || ST == 4, "");
    constexpr int TM = BM / 64, TN = BN / 128;  // 32 x 32 MFMA tiles per wave
    constexpr int NF = TM + TN;          // fragments per substep
    constexpr int NMF = TM * TN;         // MFMAs per substep
    constexpr int NRD = TM * Op<BM, A_KOUTER>::NRD + TN * Op<BN, B_KOUTER>::NRD;
    constexpr int NIA = Op<BM, A_KOUTER>::NI, NIB = Op<BN, B_KOUTER>::NI;
    constexpr int D = NIA + NIB;         // DMA instructions per wave per tile

    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int wm = (wave >> 2) * (BM / 2), wn = (wave & 3) * (BN / 4);

    uint32_t va[4], vb[4];
    int ka[4], kb[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        va[n] = n < NIA ? dma_offset<BM, A_KOUTER>(lda, wave, lane, n) : 0u;
        vb[n] = n < NIB ? dma_offset<BN, B_KOUTER>(ldb, wave, lane, n) : 0u;
        ka[n] = kb[n] = dma_kofs(wave, lane, n);
    }
    int fa_off[TM][2], fb_off[TN][2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
            fa_off[i][s] = frag_offset<BM, A_KOUTER>(wm + 32 * i, s, lane);
#pragma unroll
        for (int j = 0; j < TN; ++j)
            fb_off[j][s] = frag_offset<BN, B_KOUTER>(wn + 32 * j, s, lane);
    }

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v)
                acc[i][j][v] = 0.0f;

    const int64_t kt_n = (K + kBK - 1) / kBK, kt_full = K / kBK;
    // Descriptors end at each operand's last element: rows past M or N and
    // k rows past K read as zero without a memory access.
    auto rs_a = [&](int64_t k0) {
        return A_KOUTER ? rsrc(A + k0 * lda + m0, ((K - 1 - k0) * lda + M - m0) * 2)
                        : rsrc(A + m0 * lda + k0, ((M - 1 - m0) * lda + K - k0) * 2);
    };
    auto rs_b = [&](int64_t k0) {
        return B_KOUTER ? rsrc(B + k0 * ldb + n0, ((K - 1 - k0) * ldb + N - n0) * 2)
                        : rsrc(B + n0 * ldb + k0, ((N - 1 - n0) * ldb + K - k0) * 2);
    };
    // DMA of tile kt into stage S.  WHOLE: the tile lies inside K, so no
    // lane needs the K-inner tail mask.
    auto dma = [&](auto st, auto whole, int64_t kt) {
        constexpr int S = decltype(st)::value;
        constexpr bool WHOLE = decltype(whole)::value != 0;
        const int64_t k0 = kt * kBK;
        const __amdgpu_buffer_rsrc_t ra = rs_a(k0), rb = rs_b(k0);
#pragma unroll
        for (int n = 0; n < NIA; ++n) {
            const uint32_t o = !WHOLE && !A_KOUTER && k0 + ka[n] >= K ? kOOB : va[n];
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (ZS_LDS void *)(As[S] + (wave + kNW * n) * 1024),
                                                     16, o, 0, 0, 0);
        }
#pragma unroll
        for (int n = 0; n < NIB; ++n) {
            const uint32_t o = !WHOLE && !B_KOUTER && k0 + kb[n] >= K ? kOOB : vb[n];
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (ZS_LDS void *)(Bs[S] + (wave + kNW * n) * 1024),
                                                     16, o, 0, 0, 0);
        }
    };
    bf16x8 fa0[TM], fb0[TN], fa1[TM], fb1[TN];
    auto frags = [&](auto st, int s, bf16x8 (&fa)[TM], bf16x8 (&fb)[TN]) {
        constexpr int S = decltype(st)::value;
#pragma unroll
        for (int i = 0; i < TM; ++i)
            fa[i] = frag_read<BM, A_KOUTER>(As[S], fa_off[i][s]);
#pragma unroll
        for (int j = 0; j < TN; ++j)
            fb[j] = frag_read<BN, B_KOUTER>(Bs[S], fb_off[j][s]);
    };
    auto mma = [&](const bf16x8 (&fa)[TM], const bf16x8 (&fb)[TN], int lo, int hi) {
#pragma unroll
        for (int q = 0; q < NMF; ++q)
            if (q >= lo && q < hi)
                acc[q / TN][q % TN] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                    fa[q / TN], fb[q % TN], acc[q / TN][q % TN], 0, 0, 0);
    };
    // This wave's DMA for the tiles after `kt1` (at most two) is allowed to
    // stay in flight; everything up to tile kt1 and every LDS read is done.
    auto wait_for = [&](int64_t kt1) {
        const int64_t after = kt_n - 1 - kt1;
        if (after >= ST - 2)
            wait_vm_lgkm0<(ST - 2) * D>();
        else if (ST > 3 && after == 1)
            wait_vm_lgkm0<D>();
        else
            wait_vm_lgkm0<0>();
    };
    // Tile kt in stage S: DMA tile kt + 3 into the stage tile kt - 1 used,
    // substep 0 under the reads of substep 1, half of substep 1, wait for tile
    // kt + 1 and barrier, then the rest under the reads of tile kt + 1's
    // first substep.  STEADY: tiles kt + 1 .. kt + 3 exist and lie inside K.
    auto tile = [&](auto st, auto steady, int64_t kt) {
        constexpr int S = decltype(st)::value;
        constexpr bool STEADY = decltype(steady)::value != 0;
        constexpr int SN = (S + ST - 1) % ST, S1 = (S + 1) % ST;
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (STEADY)
            dma(IC<SN>{}, IC<1>{}, kt + ST - 1);
        else if (kt + ST - 1 < kt_n)
            dma(IC<SN>{}, IC<0>{}, kt + ST - 1);
        frags(IC<S>{}, 1, fa1, fb1);
        mma(fa0, fb0, 0, NMF);
        if constexpr (STEADY)
            seq<NF, NMF, NRD, D>();
        else
            seq<NF, NMF, NRD, 0>();
        mma(fa1, fb1, 0, NMF / 2);
        __builtin_amdgcn_sched_group_barrier(0x008, NMF / 2, 0);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (STEADY)
            wait_vm_lgkm0<(ST - 2) * D>();
        else
            wait_for(kt + 1);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        if (STEADY || kt + 1 < kt_n)
            frags(IC<S1>{}, 0, fa0, fb0);
        mma(fa1, fb1, NMF / 2, NMF);
        seq<NF, NMF / 2, NRD, 0>();
    };

    if (kt_n > 0) {
        dma(IC<0>{}, IC<0>{}, 0);
        if (kt_n > 1)
            dma(IC<1>{}, IC<0>{}, 1);
        if (ST > 3 && kt_n > 2)
            dma(IC<2>{}, IC<0>{}, 2);
        wait_for(0);
        __builtin_amdgcn_s_barrier();
        frags(IC<0>{}, 0, fa0, fb0);
        int64_t kt = 0;
        // Groups of ST tiles whose DMA targets (up to tile kt + 2 ST - 2) lie
        // inside K, then the last few tiles with checks.
        for (; kt + 2 * ST - 1 <= kt_full; kt += ST) {
            tile(IC<0>{}, IC<1>{}, kt);
            tile(IC<1>{}, IC<1>{}, kt + 1);
            tile(IC<2>{}, IC<1>{}, kt + 2);
            if constexpr (ST > 3)
                tile(IC<ST - 1>{}, IC<1>{}, kt + 3);
        }
        for (; kt < kt_n; kt += ST) {
            tile(IC<0>{}, IC<0>{}, kt);
            if (kt + 1 < kt_n)
                tile(IC<1>{}, IC<0>{}, kt + 1);
            if (kt + 2 < kt_n)
                tile(IC<2>{}, IC<0>{}, kt + 2);
            if constexpr (ST > 3)
                if (kt + 3 < kt_n)
                    tile(IC<ST - 1>{}, IC<0>{}, kt + 3);
        }
    }

    epi.template tile32<TM, TN>(acc, m0 + wm, n0 + wn, M, N, lane);
}

// Both operands K-inner (dY W^T) run on 16x16x32 MFMAs with K in 64-k stage
// pairs: a K-inner row chunk of one 32-k tile is 64 bytes, half a cache line,
// so one DMA instruction would touch 16 lines; a pair buffer holds 64 k per
// row, and each DMA instruction moves 8 whole 128-byte rows.  Two pair
// buffers per operand (128 KB).  The pair of tiles 2p, 2p + 1 is fetched at
// the start of tile 2p - 3, once the reads of pair p - 2 are done, and first
// read during tile 2p - 1: two tiles of lead, as with single stages.
// Paired against single 32-k stages: dX +10.6 %, bit-identical.
// Row r of a pair buffer holds k 0..63 of the pair as eight 16-byte chunks,
// chunk c at slot c ^ ((r >> 1) & 7); one DMA instruction moves 8 whole
// 128-byte rows.
__device__ __forceinline__ int kp_swz(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int kp_pos(int r, int c) { return r * 128 + ((c ^ kp_swz(r)) << 4); }
__device__ __forceinline__ uint32_t kp_dma_offset(int64_t ld, int wave, int lane, int n)
{
    const int r = 8 * (wave + kNW * n) + (lane >> 3), c = (lane & 7) ^ kp_swz(r);
    return (uint32_t)((r * ld + 8 * c) * 2);
}
__device__ __forceinline__ int kp_kofs(int wave, int lane, int n)
{
    const int r = 8 * (wave + kNW * n) + (lane >> 3);
    return 8 * ((lane & 7) ^ kp_swz(r));
}
constexpr int kPair = kBM * 128;  // bytes of one operand's pair buffer

template <int BM, int BN, class Epi>
__device__ __forceinline__ void gemm_tile_kp(int64_t M, int64_t N, int64_t K,
                                             const uint16_t *__restrict__ A, int64_t lda,
                                             const uint16_t *__restrict__ B, int64_t ldb,
                                             const Epi &epi, int64_t m0, int64_t n0,
                                             ZS_LDS char *A0, ZS_LDS char *A1, ZS_LDS char *B0,
                                             ZS_LDS char *B1)
{
    auto Ab = [&](auto pb) -> ZS_LDS char * {
        if constexpr (decltype(pb)::value == 0) return A0; else return A1;
    };
    auto Bb = [&](auto pb) -> ZS_LDS char * {
        if constexpr (decltype(pb)::value == 0) return B0; else return B1;
    };
    constexpr int TM = BM / 32, TN = BN / 64;
    constexpr int NF = TM + TN, NMF = TM * TN;
    constexpr int NPA = BM / (8 * kNW), NPB = BN / (8 * kNW);
    constexpr int DP = NPA + NPB;  // DMA instructions per wave per pair
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int wm = (wave >> 2) * (BM / 2), wn = (wave & 3) * (BN / 4);
    const int r16 = lane & 15, g = lane >> 4;

    uint32_t va[4], vb[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        va[n] = n < NPA ? kp_dma_offset(lda, wave, lane, n) : 0u;
        vb[n] = n < NPB ? kp_dma_offset(ldb, wave, lane, n) : 0u;
    }
    const int fa_off[2] = {kp_pos(wm + r16, g), kp_pos(wm + r16, 4 + g)};
    const int fb_off[2] = {kp_pos(wn + r16, g), kp_pos(wn + r16, 4 + g)};

    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int64_t kt_n = (K + kBK - 1) / kBK;
    const int64_t np_n = (kt_n + 1) / 2, np_full = K / (2 * kBK);
    auto dma = [&](auto pb, auto whole, int64_t p) {
        constexpr int P = decltype(pb)::value;
        constexpr bool WHOLE = decltype(whole)::value != 0;
        const int64_t k0 = p * 2 * kBK;
        const __amdgpu_buffer_rsrc_t ra = rsrc(A + m0 * lda + k0, ((M - 1 - m0) * lda + K - k0) * 2);
        const __amdgpu_buffer_rsrc_t rb = rsrc(B + n0 * ldb + k0, ((N - 1 - n0) * ldb + K - k0) * 2);
#pragma unroll
        for (int n = 0; n < NPA; ++n) {
            const uint32_t o = !WHOLE && k0 + kp_kofs(wave, lane, n) >= K ? kOOB : va[n];
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (ZS_LDS void *)(Ab(IC<P>{}) + (wave + kNW * n) * 1024), 16, o, 0, 0, 0);
        }
#pragma unroll
        for (int n = 0; n < NPB; ++n) {
            const uint32_t o = !WHOLE && k0 + kp_kofs(wave, lane, n) >= K ? kOOB : vb[n];
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (ZS_LDS void *)(Bb(IC<P>{}) + (wave + kNW * n) * 1024), 16, o, 0, 0, 0);
        }
    };
    bf16x8 fa[2][TM], fb[2][TN];
    // fragments of a tile held in pair buffer P, half H, into set F
    auto frags = [&](auto pb, auto hb, auto set) {
        constexpr int P = decltype(pb)::value, H = decltype(hb)::value, F = decltype(set)::value;
#pragma unroll
        for (int j = 0; j < TN; ++j)
            fb[F][j] = *reinterpret_cast<const ZS_LDS bf16x8 *>(Bb(IC<P>{}) + fb_off[H] + j * 2048);
#pragma unroll
        for (int i = 0; i < TM; ++i)
            fa[F][i] = *reinterpret_cast<const ZS_LDS bf16x8 *>(Ab(IC<P>{}) + fa_off[H] + i * 2048);
    };
    auto mma = [&](auto set) {
        constexpr int F = decltype(set)::value;
#pragma unroll
        for (int q = 0; q < NMF; ++q)
            acc[q / TN][q % TN] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[F][q / TN], fb[F][q % TN], acc[q / TN][q % TN], 0, 0, 0);
    };
    // Tile kt (TI = kt mod 4): odd tiles wait for tile kt + 1's pair and
    // their own fragment reads, then a barrier: after it every wave's part of
    // that pair has landed and no wave still reads the buffer the pair
    // before it used, so the DMA of the pair two ahead goes there.  Even
    // tiles only wait for their own reads: tile kt + 1 is the other half of
    // the pair already in place, and no DMA is issued, so they need no
    // barrier (paired on the dX shape: 1.022 x faster, bit-identical).
    // Read tile kt + 1's fragments under tile kt's MFMAs.
    auto tile = [&](auto ti, auto steady, int64_t kt) {
        constexpr int TI = decltype(ti)::value;
        constexpr bool STEADY = decltype(steady)::value != 0;
        constexpr bool ODD = TI & 1;
        constexpr int F = TI & 1;
        constexpr int T1 = (TI + 1) & 3;                 // tile kt + 1 mod 4
        constexpr int P1 = (T1 >> 1) & 1, H1 = T1 & 1;   // its buffer and half
        constexpr int PN = (((TI + 3) >> 1)) & 1;        // buffer of pair (kt + 3) / 2
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (ODD) {
            wait_vm_lgkm0<0>();
            __builtin_amdgcn_s_barrier();
        } else {
            wait_vm_lgkm0<DP>();
        }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (ODD) {
            const int64_t p = (kt + 3) / 2;
            if constexpr (STEADY)
                dma(IC<PN>{}, IC<1>{}, p);
            else if (p < np_n)
                dma(IC<PN>{}, IC<0>{}, p);
        }
        if (STEADY || kt + 1 < kt_n)
            frags(IC<P1>{}, IC<H1>{}, IC<F ^ 1>{});
        mma(IC<F>{});
        if constexpr (STEADY && ODD)
            seq<NF, NMF, NF, DP>();
        else
            seq<NF, NMF, NF, 0>();
    };
    if (kt_n > 0) {
        dma(IC<0>{}, IC<0>{}, 0);
        if (np_n > 1) {
            dma(IC<1>{}, IC<0>{}, 1);
            wait_vm_lgkm0<DP>();
        } else {
            wait_vm_lgkm0<0>();
        }
        __builtin_amdgcn_s_barrier();
        frags(IC<0>{}, IC<0>{}, IC<0>{});
        int64_t kt = 0;
        // steady: the pairs this group issues, (kt + 4) / 2 and (kt + 6) / 2,
        // lie inside K
        for (; (kt + 6) / 2 < np_full; kt += 4) {
            tile(IC<0>{}, IC<1>{}, kt);
            tile(IC<1>{}, IC<1>{}, kt + 1);
            tile(IC<2>{}, IC<1>{}, kt + 2);
            tile(IC<3>{}, IC<1>{}, kt + 3);
        }
        for (; kt < kt_n; kt += 4) {
            tile(IC<0>{}, IC<0>{}, kt);
            if (kt + 1 < kt_n) tile(IC<1>{}, IC<0>{}, kt + 1);
            if (kt + 2 < kt_n) tile(IC<2>{}, IC<0>{}, kt + 2);
            if (kt + 3 < kt_n) tile(IC<3>{}, IC<0>{}, kt + 3);
        }
    }
    epi.template tile16<TM, TN>(acc, m0 + wm, n0 + wn, M, N, lane);
}

// A K-inner, B K-outer (X W), 256 columns: gemm_tile with A in the 64-k pairs
// of gemm_tile_kp, whose DMA instructions move whole 128-byte rows of A where a
// 32-k stage's touch 16 half lines each.  Two pair buffers for A, four stages
// of 32 k for B, 128 KB as before; the MFMAs and their order are gemm_tile's,
// so are the results.
//
// Tile kt reads half kt % 2 of pair kt / 2.  B of tile kt + 3 goes out at the
// start of tile kt; a pair's successor in its buffer goes out behind the
// barrier of its odd tile, when every wave has read it, two tiles ahead of its
// own first read.  In order of issue: B(2p + 1), B(2p + 2), A(p + 1),
// B(2p + 3), B(2p + 4), ...; so an even tile, waiting for B(kt + 1), may leave
// B, A and B in flight, an odd one, waiting for A((kt + 1) / 2) too, two of B.
template <int BM, class Epi>
__device__ __forceinline__ void gemm_tile_ap(int64_t M, int64_t N, int64_t K,
                                             const uint16_t *__restrict__ A, int64_t lda,
                                             const uint16_t *__restrict__ B, int64_t ldb,
                                             const Epi &epi, int64_t m0, int64_t n0, ZS_LDS char *A0,
                                             ZS_LDS char *A1, ZS_LDS char *const (&Bs)[kStages])
{
    constexpr int TM = BM / 64, TN = 2, NF = TM + TN, NMF = TM * TN;
    constexpr int NRD = TM + 2 * TN;
    constexpr int NPA = BM / (8 * kNW), NIB = Op<kBN, true>::NI;

    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int wm = (wave >> 2) * (BM / 2), wn = (wave & 3) * (kBN / 4);
    const int fr = lane & 31, fh = lane >> 5;

    auto Ab = [&](auto pb) -> ZS_LDS char * {
        if constexpr (decltype(pb)::value == 0) return A0; else return A1;
    };
    uint32_t va[NPA], vb[NIB];
#pragma unroll
    for (int n = 0; n < NPA; ++n)
        va[n] = kp_dma_offset(lda, wave, lane, n);
#pragma unroll
    for (int n = 0; n < NIB; ++n)
        vb[n] = dma_offset<kBN, true>(ldb, wave, lane, n);
    // 16-byte chunk 4 h + 2 s + fh of row wm + fr; 32 rows further the swizzle
    // is the same.
    int fa_off[2][2], fb_off[TN][2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            fa_off[h][s] = kp_pos(wm + fr, 4 * h + 2 * s + fh);
#pragma unroll
        for (int j = 0; j < TN; ++j)
            fb_off[j][s] = frag_offset<kBN, true>(wn + 32 * j, s, lane);
    }

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v)
                acc[i][j][v] = 0.0f;

    const int64_t kt_n = (K + kBK - 1) / kBK, np_n = (kt_n + 1) / 2, np_full = K / (2 * kBK);
    auto dma_a = [&](auto pb, auto whole, int64_t p) {
        constexpr int P = decltype(pb)::value;
        constexpr bool WHOLE = decltype(whole)::value != 0;
        const int64_t k0 = p * 2 * kBK;
        const __amdgpu_buffer_rsrc_t ra = rsrc(A + m0 * lda + k0, ((M - 1 - m0) * lda + K - k0) * 2);
#pragma unroll
        for (int n = 0; n < NPA; ++n) {
            const uint32_t o = !WHOLE && k0 + kp_kofs(wave, lane, n) >= K ? kOOB : va[n];
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                ra, (ZS_LDS void *)(Ab(IC<P>{}) + (wave + kNW * n) * 1024), 16, o, 0, 0, 0);
        }
    };
    auto dma_b = [&](auto st, int64_t kt) {
        constexpr int S = decltype(st)::value;
        const int64_t k0 = kt * kBK;
        const __amdgpu_buffer_rsrc_t rb = rsrc(B + k0 * ldb + n0, ((K - 1 - k0) * ldb + N - n0) * 2);
#pragma unroll
        for (int n = 0; n < NIB; ++n)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (ZS_LDS void *)(Bs[S] + (wave + kNW * n) * 1024),
                                                     16, vb[n], 0, 0, 0);
    };
    bf16x8 fa0[TM], fb0[TN], fa1[TM], fb1[TN];
    auto frags = [&](auto st, auto sub, bf16x8 (&fa)[TM], bf16x8 (&fb)[TN]) {
        constexpr int S = decltype(st)::value, s = decltype(sub)::value;
#pragma unroll
        for (int i = 0; i < TM; ++i)
            fa[i] = *reinterpret_cast<const ZS_LDS bf16x8 *>(Ab(IC<(S >> 1)>{}) + fa_off[S & 1][s] + i * 4096);
#pragma unroll
        for (int j = 0; j < TN; ++j)
            fb[j] = frag_read<kBN, true>(Bs[S], fb_off[j][s]);
    };
    auto mma = [&](const bf16x8 (&fa)[TM], const bf16x8 (&fb)[TN], int lo, int hi) {
#pragma unroll
        for (int q = 0; q < NMF; ++q)
            if (q >= lo && q < hi)
                acc[q / TN][q % TN] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                    fa[q / TN], fb[q % TN], acc[q / TN][q % TN], 0, 0, 0);
    };
    auto tile = [&](auto st, auto steady, int64_t kt) {
        constexpr int S = decltype(st)::value;
        constexpr bool STEADY = decltype(steady)::value != 0, ODD = S & 1;
        constexpr int SN = (S + kStages - 1) % kStages, S1 = (S + 1) % kStages;
        // what may stay in flight at this tile's wait
        constexpr int FLY3 = ODD ? 2 * NIB : 2 * NIB + NPA, FLY2 = ODD ? NIB : NIB + NPA;
        __builtin_amdgcn_sched_barrier(0);
        if (STEADY || kt + kStages - 1 < kt_n)
            dma_b(IC<SN>{}, kt + kStages - 1);
        frags(IC<S>{}, IC<1>{}, fa1, fb1);
        mma(fa0, fb0, 0, NMF);
        seq<NF, NMF, NRD, STEADY ? NIB : 0>();
        mma(fa1, fb1, 0, NMF / 2);
        __builtin_amdgcn_sched_group_barrier(0x008, NMF / 2, 0);
        __builtin_amdgcn_sched_barrier(0);
        if (STEADY || kt + 3 < kt_n)
            wait_vm_lgkm0<FLY3>();
        else if (kt + 2 < kt_n)
            wait_vm_lgkm0<FLY2>();
        else
            wait_vm_lgkm0<0>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (ODD) {
            const int64_t p = (kt + 3) / 2;
            if constexpr (STEADY)
                dma_a(IC<(S >> 1)>{}, IC<1>{}, p);
            else if (p < np_n)
                dma_a(IC<(S >> 1)>{}, IC<0>{}, p);
        }
        if (STEADY || kt + 1 < kt_n)
            frags(IC<S1>{}, IC<0>{}, fa0, fb0);
        mma(fa1, fb1, NMF / 2, NMF);
        seq<NF, NMF / 2, NRD, STEADY && ODD ? NPA : 0>();
    };
    if (kt_n > 0) {
        dma_a(IC<0>{}, IC<0>{}, 0);
        dma_b(IC<0>{}, 0);
        if (kt_n > 1)
            dma_b(IC<1>{}, 1);
        if (kt_n > 2) {
            dma_b(IC<2>{}, 2);
            dma_a(IC<1>{}, IC<0>{}, 1);
            wait_vm_lgkm0<2 * NIB + NPA>();
        } else {
            wait_vm_lgkm0<0>();
        }
        __builtin_amdgcn_s_barrier();
        frags(IC<0>{}, IC<0>{}, fa0, fb0);
        int64_t kt = 0;
        // steady: the pairs this group issues, (kt + 4) / 2 and (kt + 6) / 2,
        // lie inside K
        for (; (kt + 6) / 2 < np_full; kt += kStages) {
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

}  // namespace
}  // namespace zs
