// Around the tiles of gemm_tile.h, for kernels with an epilogue of their own: the
// blocks' LDS, each wave's corner of it once the K loop is done, and which tile a
// block computes.
#pragma once

#include "gemm_tile.h"
#include "products.h"

namespace zs {
namespace {

// A wave's LDS traffic is in order; this keeps the compiler to that order
// where one lane reads what another wrote.
__device__ __forceinline__ void wave_lds_order()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The wave's corner of the K loop's LDS: array w of the eight stages.
#define ZS_STAGES(BM_, BN_)                                                                        \
    __shared__ __attribute__((aligned(1024))) char a0[BM_ * 64], a1[BM_ * 64], a2[BM_ * 64],       \
        a3[BM_ * 64];                                                                              \
    __shared__ __attribute__((aligned(1024))) char b0[BN_ * 64], b1[BN_ * 64], b2[BN_ * 64],       \
        b3[BN_ * 64];                                                                              \
    ZS_LDS char *const As[kStages] = {(ZS_LDS char *)a0, (ZS_LDS char *)a1, (ZS_LDS char *)a2,     \
                                      (ZS_LDS char *)a3};                                          \
    ZS_LDS char *const Bs[kStages] = {(ZS_LDS char *)b0, (ZS_LDS char *)b1, (ZS_LDS char *)b2,     \
                                      (ZS_LDS char *)b3}

// By value: an array of LDS addresses indexed by the wave would have to exist
// in memory.
__device__ __forceinline__ ZS_LDS float *corner(ZS_LDS char *a0, ZS_LDS char *a1, ZS_LDS char *a2, ZS_LDS char *a3,
                                                ZS_LDS char *b0, ZS_LDS char *b1, ZS_LDS char *b2, ZS_LDS char *b3)
{
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint32_t p = (uint32_t)(uintptr_t)a0;
    p = w == 1 ? (uint32_t)(uintptr_t)a1 : p;
    p = w == 2 ? (uint32_t)(uintptr_t)a2 : p;
    p = w == 3 ? (uint32_t)(uintptr_t)a3 : p;
    p = w == 4 ? (uint32_t)(uintptr_t)b0 : p;
    p = w == 5 ? (uint32_t)(uintptr_t)b1 : p;
    p = w == 6 ? (uint32_t)(uintptr_t)b2 : p;
    p = w == 7 ? (uint32_t)(uintptr_t)b3 : p;
    return (ZS_LDS float *)p;
}
#define ZS_CORNER                                                                                  \
    corner((ZS_LDS char *)a0, (ZS_LDS char *)a1, (ZS_LDS char *)a2, (ZS_LDS char *)a3,             \
           (ZS_LDS char *)b0, (ZS_LDS char *)b1, (ZS_LDS char *)b2, (ZS_LDS char *)b3)

#define ZS_PAIRS(BM_, BN_)                                                                         \
    __shared__ __attribute__((aligned(1024))) char pa0[BM_ * 128], pa1[BM_ * 128];                 \
    __shared__ __attribute__((aligned(1024))) char pb0[BN_ * 128], pb1[BN_ * 128];

// Two waves to an array, each its half.
#define ZS_CORNER_KP(HALF)                                                                         \
    corner((ZS_LDS char *)pa0, (ZS_LDS char *)pa0 + (HALF), (ZS_LDS char *)pa1,                    \
           (ZS_LDS char *)pa1 + (HALF), (ZS_LDS char *)pb0, (ZS_LDS char *)pb0 + (HALF),           \
           (ZS_LDS char *)pb1, (ZS_LDS char *)pb1 + (HALF))
#define ZS_P (ZS_LDS char *)pa0, (ZS_LDS char *)pa1, (ZS_LDS char *)pb0, (ZS_LDS char *)pb1

// Block b of n_big + 2 (T - n_big): a whole tile, or a half of BM / 2 rows
// (as gemm.hip's kernels place them).
template <int BM, int BN>
__device__ __forceinline__ bool place(int tiles_m, int tiles_n, int n_big, int64_t &m0, int64_t &n0)
{
    const int b = blockIdx.x;
    int tm, tn;
    if (b < n_big) {
        grouped(xcd_order(b, n_big), tiles_m, tiles_n, tm, tn);
        m0 = (int64_t)tm * BM;
        n0 = (int64_t)tn * BN;
        return true;
    }
    const int h = xcd_order(b - n_big, (int)gridDim.x - n_big);
    grouped(n_big + h / 2, tiles_m, tiles_n, tm, tn);
    m0 = (int64_t)tm * BM + (h & 1) * (BM / 2);
    n0 = (int64_t)tn * BN;
    return false;
}

struct Grid {
    int tm, tn, n_big;
    dim3 grid;
};

// Tiles of bm x bn; with `halves`, a last wave of at most half the CUs runs
// as twice as many half tiles.
inline Grid tiles(int64_t M, int64_t N, int bm, int bn, bool halves)
{
    Grid g;
    const int64_t tm = (M + bm - 1) / bm, tn = (N + bn - 1) / bn, T = tm * tn, P = cu_count();
    const int64_t rem = T % P;
    const int64_t big = halves && rem > 0 && rem <= P / 2 ? T - rem : T;
    g.tm = (int)tm;
    g.tn = (int)tn;
    g.n_big = (int)big;
    g.grid = dim3((unsigned)(big + 2 * (T - big)));
    return g;
}

// 128 x 128 tiles where 256 x 256 ones would not fill half the CUs.
inline bool small_tiles(int64_t M, int64_t N)
{
    const int64_t T = ((M + kBM - 1) / kBM) * ((N + kBN - 1) / kBN);
    return 2 * T <= cu_count();
}

}  // namespace
}  // namespace zs
