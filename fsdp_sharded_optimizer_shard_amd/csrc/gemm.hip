// bf16 GEMM on MFMA (gfx950) and a bf16 transpose: the dense contractions of
// a hand-written FSDP linear layer ("DP, ZeRO-1/2/3, FSDP" notes, follow-up
// on writing one FSDP linear layer by hand).
//
//   zero_gemm_bf16:     C[i][j] = sum_k a(i, k) b(j, k), fp32 accumulation, C
//                       fp32 or bf16 (round to nearest even).  Each operand is
//                       stored either K-inner (A as M x K, B as N x K) or
//                       K-outer (A as K x M, B as K x N), so X W, dY W^T and
//                       X^T dY all run without a separate transpose.
//   zero_gemm_bf16_nt:  the K-inner / K-inner case.
//   zero_transpose_bf16: dst[c][r] = src[r][c].
//
// GEMM tiling (the tile functions are in gemm_tile.h).  A 512-thread block (8 waves, two per SIMD) owns a 256 x 256
// tile of C; each wave owns 128 x 64 as 4 x 2 tiles of
// v_mfma_f32_32x32x16_bf16 (128 fp32 accumulators per lane), so while one
// wave of a SIMD waits on its fragment reads the other issues MFMAs.  K
// advances 32 at a time through four LDS stages of 256 x 32 bf16 per
// operand (128 KB in all).
//
// Loads.  Operands go from HBM straight into LDS with buffer_load ... lds
// (16 bytes per lane, 1 KB per wave instruction): no register staging and
// no LDS write instructions.  The DMA of tile k + 3 is issued at the start
// of tile k, into the stage tile k - 1 has just released, so three tiles of
// loads are in flight.  Each block's buffer descriptors end at the
// operand's last element, so rows past M or N and k past K read as zero
// without touching memory.
//
// LDS layouts.  A K-inner stage has 64-byte rows (32 k); 16-byte chunk c of
// row r sits at slot c ^ ((r >> 2) & 3), which keeps the fragment reads
// (ds_read_b128) free of bank conflicts.  A K-outer stage is k-major (one
// 2R-byte row per k); its 32-byte units are permuted per k row (unit_pos), and a
// fragment is two ds_read_b64_tr_b16 that transpose 4 x 4 blocks of 16-bit
// values across each 16-lane group.  A DMA lane's global address is chosen
// so that it lands in the swizzled slot.  Both layouts read without bank
// conflicts (rocprofv3 SQ_LDS_BANK_CONFLICT reads 0).
//
// Pipeline per K tile of 32 (two MFMA substeps of 16): DMA of tile k + 3;
// substep 0 under the fragment reads of substep 1; half of substep 1; wait
// for this wave's DMA of tile k + 1 (two tiles may stay in flight) and its
// LDS reads, then one barrier; the rest of substep 1 under the reads of
// tile k + 1's first substep.  sched_group_barrier fixes that interleave.
// Measured against the previous design (register staging, two 64-k LDS
// buffers, one tile ahead), paired on the Mistral-7B MLP shapes with random
// operands: dX +8.5 %, forward +4.2 %, dW +6.7 %, 8192^3 +9.1 %; then eight
// waves instead of four (128 x 128 each): dX +4.9 %, forward +15 %, dW +9 %;
// a 2 x 4 wave grid (128 x 64 per wave) rather than 4 x 2 adds about 1 %
// and needs no register spills.  Every step gave bit-identical results.
//
// Tile order.  Block b runs on XCD b % 8; each XCD gets a contiguous range of
// tiles, walked 4 tile rows at a time, so the blocks that share an L2 share
// A rows and B columns.
//
// Both operands K-inner (dY W^T): 16x16x32 MFMAs and 64-k stage pairs
// (gemm_tile_kp), so that every DMA instruction moves whole cache
// lines; a pair lands every second tile, so only those tiles need a
// barrier.
//
// MFMA 32x32x16 bf16 lane layout (checked on the device against an exact
// CPU product): lane l holds A row (l % 32), k = 8 (l / 32) .. +7, and B
// column (l % 32) at the same k; accumulator v of lane l is row
// 8 (v / 4) + 4 (l / 32) + (v % 4), column l % 32.
#include <hip/hip_runtime.h>

#include <atomic>
#include <climits>
#include <cstdint>

#include "gemm_tile.h"
#include "products.h"

namespace zs {
namespace {

// Blocks [0, n_big) compute whole 256 x 256 tiles (big tiles 0 .. n_big-1 in
// grouped order); the remaining blocks split the last big tiles into
// 128 x 256 halves, two blocks per tile, so a partial last wave of big
// tiles becomes a wave of half-length work.
template <bool A_KOUTER, bool B_KOUTER, bool OUT_BF16>
__global__ __launch_bounds__(kGT) void gemm_kernel(int64_t M, int64_t N, int64_t K,
                                                   const uint16_t *__restrict__ A, int64_t lda,
                                                   const uint16_t *__restrict__ B, int64_t ldb,
                                                   void *__restrict__ C, int64_t ldc, int tiles_m,
                                                   int tiles_n, int n_big)
{
    // One array per stage and operand, so the compiler can tell the LDS a
    // DMA writes from the LDS the fragment reads use.
    __shared__ __attribute__((aligned(1024))) char a0[kStage], a1[kStage], a2[kStage], a3[kStage];
    __shared__ __attribute__((aligned(1024))) char b0[kStage], b1[kStage], b2[kStage], b3[kStage];
    ZS_LDS char *const As[kStages] = {(ZS_LDS char *)a0, (ZS_LDS char *)a1, (ZS_LDS char *)a2,
                                      (ZS_LDS char *)a3};
    ZS_LDS char *const Bs[kStages] = {(ZS_LDS char *)b0, (ZS_LDS char *)b1, (ZS_LDS char *)b2,
                                      (ZS_LDS char *)b3};
    const PlainEpi<OUT_BF16> epi{C, ldc};
    const int b = blockIdx.x;
    int tm, tn;
    if (b < n_big) {
        grouped(xcd_order(b, n_big), tiles_m, tiles_n, tm, tn);
        gemm_tile<kBM, kBN, A_KOUTER, B_KOUTER>(M, N, K, A, lda, B, ldb, epi, (int64_t)tm * kBM,
                                                (int64_t)tn * kBN, As, Bs);
    } else {
        const int h = xcd_order(b - n_big, (int)gridDim.x - n_big);
        grouped(n_big + h / 2, tiles_m, tiles_n, tm, tn);
        const int64_t hm0 = (int64_t)tm * kBM + (h & 1) * (kBM / 2);
        gemm_tile<kBM / 2, kBN, A_KOUTER, B_KOUTER>(M, N, K, A, lda, B, ldb, epi, hm0,
                                                    (int64_t)tn * kBN, As, Bs);
    }
}

// The both-K-inner order: gemm_tile_kp with its pair buffers, whole tiles and
// half tiles as in gemm_kernel.
template <bool OUT_BF16>
__global__ __launch_bounds__(kGT) void gemm_kernel_kp(int64_t M, int64_t N, int64_t K,
                                                      const uint16_t *__restrict__ A, int64_t lda,
                                                      const uint16_t *__restrict__ B, int64_t ldb,
                                                      void *__restrict__ C, int64_t ldc, int tiles_m,
                                                      int tiles_n, int n_big)
{
    __shared__ __attribute__((aligned(1024))) char pa0[kPair], pa1[kPair];
    __shared__ __attribute__((aligned(1024))) char pb0[kPair], pb1[kPair];
    const PlainEpi<OUT_BF16> epi{C, ldc};
    const int b = blockIdx.x;
    int tm, tn;
    if (b < n_big) {
        grouped(xcd_order(b, n_big), tiles_m, tiles_n, tm, tn);
        gemm_tile_kp<kBM, kBN>(M, N, K, A, lda, B, ldb, epi, (int64_t)tm * kBM, (int64_t)tn * kBN,
                               (ZS_LDS char *)pa0, (ZS_LDS char *)pa1, (ZS_LDS char *)pb0,
                               (ZS_LDS char *)pb1);
    } else {
        const int h = xcd_order(b - n_big, (int)gridDim.x - n_big);
        grouped(n_big + h / 2, tiles_m, tiles_n, tm, tn);
        const int64_t hm0 = (int64_t)tm * kBM + (h & 1) * (kBM / 2);
        gemm_tile_kp<kBM / 2, kBN>(M, N, K, A, lda, B, ldb, epi, hm0, (int64_t)tn * kBN,
                                   (ZS_LDS char *)pa0, (ZS_LDS char *)pa1, (ZS_LDS char *)pb0,
                                   (ZS_LDS char *)pb1);
    }
}

// 64 x 64 tiles through LDS (one padding column against bank conflicts):
// reads along src rows and writes along dst rows are both coalesced.
constexpr int kTT = 64;
__global__ __launch_bounds__(256) void transpose_kernel(int64_t rows, int64_t cols,
                                                        const uint16_t *__restrict__ src,
                                                        int64_t lds, uint16_t *__restrict__ dst,
                                                        int64_t ldd)
{
    __shared__ uint16_t t[kTT][kTT + 2];
    const int64_t r0 = (int64_t)blockIdx.y * kTT, c0 = (int64_t)blockIdx.x * kTT;
    const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
    for (int i = ty; i < kTT; i += 4) {
        const int64_t r = r0 + i, c = c0 + tx;
        t[i][tx] = (r < rows && c < cols) ? src[r * lds + c] : (uint16_t)0;
    }
    __syncthreads();
    for (int i = ty; i < kTT; i += 4) {
        const int64_t c = c0 + i, r = r0 + tx;  // dst row c, column r
        if (c < cols && r < rows)
            dst[c * ldd + r] = t[tx][i];
    }
}

// Fills rows [r0, r1) x cols of an fp32 matrix with zeros (a kernel, so it
// is safe inside captured graphs).
__global__ __launch_bounds__(256) void zero_rows_kernel(float *p, int64_t ld, int64_t r0,
                                                        int64_t r1, int64_t cols)
{
    const int64_t n = (r1 - r0) * cols;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n;
         i += (int64_t)gridDim.x * 256)
        p[(r0 + i / cols) * ld + i % cols] = 0.0f;
}

bool a16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

zero_status launched(const char *what)
{
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return fail(ZERO_ERR_HIP, "%s launch failed: %s", what, hipGetErrorString(e));
    return ZERO_OK;
}

}  // namespace

// Compute units of the current device, cached per device (atomics: calls
// may come from several host threads at once).
int cu_count()
{
    static std::atomic<int> cache[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess)
        dev = -1;
    if (dev >= 0 && dev < 64) {
        const int c = cache[dev].load(std::memory_order_relaxed);
        if (c > 0)
            return c;
    }
    int n = 0;
    if (dev < 0 || hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) !=
                       hipSuccess || n <= 0)
        n = 256;
    if (dev >= 0 && dev < 64)
        cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

zero_status zero_rows_fill(float *p, int64_t ld, int64_t r0, int64_t r1, int64_t cols,
                           hipStream_t s)
{
    if (r1 <= r0 || cols <= 0)
        return ZERO_OK;
    const int64_t n = (r1 - r0) * cols;
    int64_t grid = (n + 255) / 256;
    grid = grid > 65536 ? 65536 : grid;
    (void)hipGetLastError();
    hipLaunchKernelGGL(zero_rows_kernel, dim3((unsigned)grid), dim3(256), 0, s, p, ld, r0, r1,
                       cols);
    return launched("zero_rows");
}

}  // namespace zs

namespace zs {

// Every argument check of zero_gemm_bf16, with nothing launched; composite
// calls (the FSDP linear layer) run it for each of their GEMMs before their
// first launch.
zero_status gemm_check(int64_t M, int64_t N, int64_t K, const uint16_t *A, int64_t lda,
                       int32_t a_order, const uint16_t *B, int64_t ldb, int32_t b_order,
                       const void *C, int64_t ldc, int32_t c_dtype)
{
    if (M < 0 || N < 0 || K < 0)
        return fail(ZERO_ERR_INVALID_ARG, "negative GEMM size");
    if ((a_order != ZERO_K_INNER && a_order != ZERO_K_OUTER) ||
        (b_order != ZERO_K_INNER && b_order != ZERO_K_OUTER))
        return fail(ZERO_ERR_INVALID_ARG, "unknown operand order (%d, %d)", a_order, b_order);
    if (c_dtype != ZERO_BF16 && c_dtype != ZERO_FP32)
        return fail(ZERO_ERR_INVALID_ARG, "unknown C dtype %d", c_dtype);
    if (M == 0 || N == 0)
        return ZERO_OK;
    if (!A || !B || !C)
        return fail(ZERO_ERR_INVALID_ARG, "A, B and C are required");
    const bool ao = a_order == ZERO_K_OUTER, bo = b_order == ZERO_K_OUTER;
    if (K % 8 || lda % 8 || ldb % 8)
        return fail(ZERO_ERR_UNSUPPORTED, "GEMM needs K, lda and ldb multiples of 8");
    if ((ao && M % 8) || (bo && N % 8))
        return fail(ZERO_ERR_UNSUPPORTED, "a K-outer operand needs its M or N a multiple of 8");
    if (lda < (ao ? M : K) || ldb < (bo ? N : K) || ldc < N)
        return fail(ZERO_ERR_INVALID_ARG, "leading dimension too small (lda %lld, ldb %lld, "
                    "ldc %lld)", (long long)lda, (long long)ldb, (long long)ldc);
    // The kernel reads a K-inner operand's 256-row panel (at most 510 ld + 64
    // bytes from its start) and a K-outer operand's 32 k rows (at most
    // 62 ld + 512) through 32-bit buffer offsets below 2^31.
    const int64_t ki_max = int64_t(1) << 22, ko_max = int64_t(1) << 25;
    if (lda > (ao ? ko_max : ki_max) || ldb > (bo ? ko_max : ki_max))
        return fail(ZERO_ERR_UNSUPPORTED, "leading dimension too large for 32-bit operand offsets "
                    "(lda %lld, ldb %lld; K-inner at most %lld, K-outer at most %lld)",
                    (long long)lda, (long long)ldb, (long long)ki_max, (long long)ko_max);
    // The dispatch counts the grid in work-items, 32 bits wide, and the grid
    // has up to two blocks per tile.
    const int64_t tm = (M + zs::kBM - 1) / zs::kBM, tn = (N + zs::kBN - 1) / zs::kBN;
    constexpr int64_t kMaxTiles = int64_t(0xffffffffu) / (2 * zs::kGT);
    if (tm > kMaxTiles / tn)
        return fail(ZERO_ERR_UNSUPPORTED, "too many GEMM tiles for one launch (%lld x %lld)",
                    (long long)tm, (long long)tn);
    if (!zs::a16(A) || !zs::a16(B))
        return fail(ZERO_ERR_ALIGNMENT, "A and B must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(C) % (c_dtype == ZERO_BF16 ? 2 : 4))
        return fail(ZERO_ERR_ALIGNMENT, "C is misaligned");
    return ZERO_OK;
}

// The launch of zero_gemm_bf16 on checked arguments.  With both operands
// K-outer K may be any number: k rows past K are outside both descriptors.
zero_status gemm_run(int64_t M, int64_t N, int64_t K, const uint16_t *A, int64_t lda, int32_t a_order,
                     const uint16_t *B, int64_t ldb, int32_t b_order, void *C, int64_t ldc,
                     int32_t c_dtype, hipStream_t s)
{
    if (M == 0 || N == 0)
        return ZERO_OK;
    const bool ao = a_order == ZERO_K_OUTER, bo = b_order == ZERO_K_OUTER;
    const int64_t tm = (M + kBM - 1) / kBM, tn = (N + kBN - 1) / kBN;
    // One block per CU at a time (128 KB of LDS).  A last wave of at most
    // half the CUs runs as twice as many half tiles.
    const int64_t T = tm * tn, P = cu_count();
    const int64_t rem = T % P;
    const int64_t n_big = rem > 0 && rem <= P / 2 ? T - rem : T;
    const dim3 grid((unsigned)(n_big + 2 * (T - n_big))), block(kGT);
    const int code = (ao ? 1 : 0) | (bo ? 2 : 0) | (c_dtype == ZERO_BF16 ? 4 : 0);
    (void)hipGetLastError();
#define ZS_GEMM(AO, BO, BF)                                                                      \
    hipLaunchKernelGGL((gemm_kernel<AO, BO, BF>), grid, block, 0, s, M, N, K, A, lda, B, ldb, \
                       C, ldc, (int)tm, (int)tn, (int)n_big)
    switch (code) {
    case 0:
        hipLaunchKernelGGL((gemm_kernel_kp<false>), grid, block, 0, s, M, N, K, A, lda, B, ldb,
                           C, ldc, (int)tm, (int)tn, (int)n_big);
        break;
    case 4:
        hipLaunchKernelGGL((gemm_kernel_kp<true>), grid, block, 0, s, M, N, K, A, lda, B, ldb,
                           C, ldc, (int)tm, (int)tn, (int)n_big);
        break;
    case 1: ZS_GEMM(true, false, false); break;
    case 2: ZS_GEMM(false, true, false); break;
    case 3: ZS_GEMM(true, true, false); break;
    case 5: ZS_GEMM(true, false, true); break;
    case 6: ZS_GEMM(false, true, true); break;
    default: ZS_GEMM(true, true, true); break;
    }
#undef ZS_GEMM
    return launched("gemm");
}

}  // namespace zs

extern "C" {

zero_status zero_gemm_bf16(int64_t M, int64_t N, int64_t K, const uint16_t *A, int64_t lda,
                           int32_t a_order, const uint16_t *B, int64_t ldb, int32_t b_order,
                           void *C, int64_t ldc, int32_t c_dtype, void *stream)
{
    const zero_status st = zs::gemm_check(M, N, K, A, lda, a_order, B, ldb, b_order, C, ldc,
                                          c_dtype);
    if (st != ZERO_OK)
        return st;
    return zs::gemm_run(M, N, K, A, lda, a_order, B, ldb, b_order, C, ldc, c_dtype,
                        static_cast<hipStream_t>(stream));
}

zero_status zero_gemm_bf16_nt(int64_t M, int64_t N, int64_t K, const uint16_t *A, int64_t lda,
                              const uint16_t *B, int64_t ldb, void *C, int64_t ldc,
                              int32_t c_dtype, void *stream)
{
    return zero_gemm_bf16(M, N, K, A, lda, ZERO_K_INNER, B, ldb, ZERO_K_INNER, C, ldc, c_dtype,
                          stream);
}

zero_status zero_transpose_bf16(int64_t rows, int64_t cols, const uint16_t *src, int64_t lds,
                                uint16_t *dst, int64_t ldd, void *stream)
{
    using zs::fail;
    if (rows < 0 || cols < 0)
        return fail(ZERO_ERR_INVALID_ARG, "negative transpose size");
    if (rows == 0 || cols == 0)
        return ZERO_OK;
    if (!src || !dst || lds < cols || ldd < rows)
        return fail(ZERO_ERR_INVALID_ARG, "transpose needs src, dst, lds >= cols, ldd >= rows");
    if (reinterpret_cast<uintptr_t>(src) % 2 || reinterpret_cast<uintptr_t>(dst) % 2)
        return fail(ZERO_ERR_ALIGNMENT, "transpose buffers are misaligned");
    if ((rows + zs::kTT - 1) / zs::kTT > 65535 ||
        (cols + zs::kTT - 1) / zs::kTT > int64_t(0xffffffffu) / 256)
        return fail(ZERO_ERR_UNSUPPORTED, "transpose too large for one launch");
    const dim3 grid((unsigned)((cols + zs::kTT - 1) / zs::kTT),
                    (unsigned)((rows + zs::kTT - 1) / zs::kTT));
    (void)hipGetLastError();
    hipLaunchKernelGGL(zs::transpose_kernel, grid, dim3(256), 0, static_cast<hipStream_t>(stream),
                       rows, cols, src, lds, dst, ldd);
    return zs::launched("transpose");
}

}  // extern "C"
