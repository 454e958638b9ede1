// The products of gemm.hip and layer.hip as the library's own composite calls
// use them.  Not part of the C ABI.
#pragma once

#include <hip/hip_runtime_api.h>

#include "internal.h"

namespace zs {

// Compute units of the current device.
int cu_count();

// The products behind the C entry points.  A *_check makes every argument
// check of its call and launches nothing, so that a composite call can check
// all of its steps before the first launch; a *_run launches on arguments
// that were checked.
zero_status gemm_check(int64_t M, int64_t N, int64_t K, const uint16_t *A, int64_t lda,
                       int32_t a_order, const uint16_t *B, int64_t ldb, int32_t b_order,
                       const void *C, int64_t ldc, int32_t c_dtype);
// An operand for gemm_check: one that is never read, as in a product of K = 0, may
// be NULL, which an empty tensor's address is; gemm_check wants an address.
inline const uint16_t *operand(const uint16_t *p, bool read)
{
    alignas(16) static const uint16_t unread[8] = {};
    return p || read ? p : unread;
}
zero_status gemm_run(int64_t M, int64_t N, int64_t K, const uint16_t *A, int64_t lda, int32_t a_order,
                     const uint16_t *B, int64_t ldb, int32_t b_order, void *C, int64_t ldc,
                     int32_t c_dtype, hipStream_t s);

// Fills rows [r0, r1) x cols of an fp32 matrix with zeros.
zero_status zero_rows_fill(float *p, int64_t ld, int64_t r0, int64_t r1, int64_t cols,
                           hipStream_t s);

zero_status epilogue_check(int64_t M, int64_t N, const void *A, const void *B, const void *C, int64_t ldc,
                           int32_t c_dtype, const zero_epilogue *ep, const int64_t *offsets);
zero_status epilogue_gemm_run(int64_t M, int64_t N, int64_t K, const uint16_t *A, int64_t lda,
                              int32_t a_order, const uint16_t *B, int64_t ldb, int32_t b_order, void *C,
                              int64_t ldc, int32_t c_dtype, const zero_epilogue *ep, hipStream_t s);

zero_status act_backward_check(int64_t rows, int64_t cols, const void *dy, int64_t ldy, int32_t dy_dtype,
                               int32_t act, const zero_saved *preact, const uint16_t *dz, int64_t ldz,
                               const float *dbias, const float *workspace, int64_t n_workspace);
zero_status act_backward_run(int64_t rows, int64_t cols, const void *dy, int64_t ldy, int32_t dy_dtype,
                             int32_t act, const zero_saved *preact, uint16_t *dz, int64_t ldz, float *dbias,
                             float *workspace, hipStream_t s);

zero_status gemm_saved_check(int64_t M, int64_t N, int64_t K, const zero_saved *A, const uint16_t *B,
                             int64_t ldb, const void *C, int64_t ldc, int32_t c_dtype);
zero_status gemm_saved_run(int64_t M, int64_t N, int64_t K, const zero_saved *A, const uint16_t *B,
                           int64_t ldb, void *C, int64_t ldc, int32_t c_dtype, hipStream_t s);

zero_status grouped_rows_check(int32_t n_groups, const int64_t *offsets, int64_t rows, int64_t N, int64_t K,
                               const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb,
                               int32_t b_order, int64_t stride_b, const void *C, int64_t ldc,
                               int32_t c_dtype, const zero_epilogue *ep);
zero_status grouped_rows_run(int32_t n_groups, const int64_t *offsets, int64_t rows, int64_t N, int64_t K,
                             const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb,
                             int32_t b_order, int64_t stride_b, void *C, int64_t ldc, int32_t c_dtype,
                             const zero_epilogue *ep, hipStream_t s);
zero_status grouped_depth_check(int32_t n_groups, const int64_t *offsets, int64_t rows, int64_t M, int64_t N,
                                const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb,
                                const void *C, int64_t ldc, int64_t stride_c, int32_t c_dtype);
zero_status grouped_depth_run(int32_t n_groups, const int64_t *offsets, int64_t rows, int64_t M, int64_t N,
                              const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb, void *C,
                              int64_t ldc, int64_t stride_c, int32_t c_dtype, hipStream_t s);

// The cross entropy of a linear head (zero_linear_xent_*).
zero_status xent_forward_check(int64_t rows, int64_t vocab, int64_t hidden, const uint16_t *x, int64_t ldx,
                               const uint16_t *w, int64_t ldw, int32_t w_order, const int64_t *targets,
                               const float *loss, const float *lse, const float *workspace, int64_t n_workspace);
zero_status xent_forward_run(int64_t rows, int64_t vocab, int64_t hidden, const uint16_t *x, int64_t ldx,
                             const uint16_t *w, int64_t ldw, int32_t w_order, const int64_t *targets, float *loss,
                             float *lse, float *workspace, hipStream_t s);
zero_status xent_backward_check(int64_t rows, int64_t vocab, int64_t hidden, const uint16_t *x, int64_t ldx,
                                const uint16_t *w, int64_t ldw, int32_t w_order, const int64_t *targets,
                                const float *lse, const float *dloss, const void *dx, int64_t lddx, int32_t dx_dtype,
                                const void *dw, int64_t lddw, int32_t dw_dtype, int64_t piece, const float *workspace,
                                int64_t n_workspace);
zero_status xent_backward_run(int64_t rows, int64_t vocab, int64_t hidden, const uint16_t *x, int64_t ldx,
                              const uint16_t *w, int64_t ldw, int32_t w_order, const int64_t *targets,
                              const float *lse, const float *dloss, void *dx, int64_t lddx, int32_t dx_dtype, void *dw,
                              int64_t lddw, int32_t dw_dtype, int64_t piece, float *workspace, hipStream_t s);

}  // namespace zs
