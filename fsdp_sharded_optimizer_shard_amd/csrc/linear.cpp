// A hand-written FSDP linear layer for one rank ("DP, ZeRO-1/2/3, FSDP"
// notes, follow-up on writing one FSDP linear layer by hand): every rank
// stores 1/N of the rows of W; forward all-gathers the full W and computes
// X W for the local batch; backward all-gathers W again, computes dX and the
// full-shape dW locally; the reduce-scatter of dW over the ranks is
// zero_reduce_shard on the N ranks' dW buffers.
//
// W is unit `unit` of a row layout (zero_shard_init_rows) with rows =
// in_features and cols = out_features, so Y = X W takes (batch x in) to
// (batch x out).  The contractions run on the MFMA GEMM, which reads each
// operand in place, contiguous along K or along its rows, so no transposed
// copy is made.  The batch is the K of the dW product, hence the GEMM's
// multiple-of-8 rule on it.
#include <hip/hip_runtime.h>

#include <initializer_list>

#include "checks.h"
#include "products.h"

namespace {

using zs::data_of;
using zs::is_one_of;
using zs::scales_of;

struct Dims {
    int64_t in, out, in_pad;
};

zero_status layer_dims(const zero_layout *L, int32_t unit, Dims *d)
{
    if (!L)
        return zs::fail(ZERO_ERR_INVALID_ARG, "layout is NULL");
    if (unit < 0 || unit >= L->n_units)
        return zs::fail(ZERO_ERR_INVALID_ARG, "unit %d outside [0, %d)", unit, L->n_units);
    d->out = L->cols[unit];
    d->in = L->numel[unit] / d->out;
    d->in_pad = L->padded[unit] / d->out;
    return ZERO_OK;
}

// The shards the gather reads: every one present and 2-byte aligned (the
// gather's own checks), so that a layer call fails before its first launch.
zero_status check_shards(const zero_layout *L, const uint16_t *const *w_shards)
{
    for (int32_t q = 0; q < L->parts; ++q) {
        if (!w_shards[q])
            return zs::fail(ZERO_ERR_INVALID_ARG, "W shard of rank %d is NULL", q);
        if (reinterpret_cast<uintptr_t>(w_shards[q]) % 2)
            return zs::fail(ZERO_ERR_ALIGNMENT, "W shard of rank %d is misaligned", q);
    }
    return ZERO_OK;
}

// No result over a shard, which is some rank's weight after the call too.
zero_status check_results(const zero_layout *L, const uint16_t *const *w_shards,
                          std::initializer_list<const void *> results)
{
    for (int32_t q = 0; q < L->parts; ++q)
        if (is_one_of(w_shards[q], results))
            return zs::fail(ZERO_ERR_INVALID_ARG, "a result must not lie over the W shard of rank %d", q);
    return ZERO_OK;
}

// An expert unit's dimensions: in is one expert's, in_pad the whole unit's
// padded rows.
zero_status expert_dims(const zero_layout *L, int32_t unit, int32_t n_experts, Dims *d)
{
    const zero_status st = layer_dims(L, unit, d);
    if (st != ZERO_OK)
        return st;
    if (n_experts < 1 || d->in % n_experts)
        return zs::fail(ZERO_ERR_INVALID_ARG, "unit %d has %lld rows, not a multiple of %d experts",
                        unit, (long long)d->in, n_experts);
    d->in /= n_experts;
    if (d->in % 8 || d->out % 8)
        return zs::fail(ZERO_ERR_UNSUPPORTED, "in_features and out_features must be "
                        "multiples of 8");
    return ZERO_OK;
}

// The gather writes w_full before a forward product reads anything else; what
// the product writes over w_full is its own checks' to find, over a shard not.
zero_status check_gathered(const zero_layout *L, const uint16_t *const *w_shards, const uint16_t *w_full,
                           const uint16_t *x, const int64_t *offsets, const zero_epilogue *ep, const void *y)
{
    if (is_one_of(w_full, {x, offsets, ep ? ep->bias : nullptr, ep ? ep->residual : nullptr}))
        return zs::fail(ZERO_ERR_INVALID_ARG, "w_full must not lie where the call reads something else");
    const zero_saved *z = ep ? ep->preact : nullptr, *o = ep ? ep->output : nullptr;
    return check_results(L, w_shards, {y, data_of(z), scales_of(z), data_of(o), scales_of(o)});
}

}  // namespace

extern "C" {

zero_status zero_fsdp_linear_forward(const zero_layout *L, int32_t unit,
                                     const uint16_t *const *w_shards, int64_t batch,
                                     const uint16_t *x, uint16_t *w_full, void *y,
                                     int32_t y_dtype, void *stream)
{
    Dims d;
    zero_status st = layer_dims(L, unit, &d);
    if (st != ZERO_OK)
        return st;
    if (!w_shards || !x || !w_full || !y || batch < 0)
        return zs::fail(ZERO_ERR_INVALID_ARG, "w_shards, x, w_full, y and batch >= 0 are "
                        "required");
    if ((st = check_shards(L, w_shards)) != ZERO_OK)
        return st;
    if (d.in % 8 || d.out % 8)
        return zs::fail(ZERO_ERR_UNSUPPORTED, "in_features and out_features must be "
                        "multiples of 8");
    // every check before the first launch: the GEMM's too
    if ((st = zs::gemm_check(batch, d.out, d.in, x, d.in, ZERO_K_INNER, w_full, d.out,
                             ZERO_K_OUTER, y, d.out, y_dtype)) != ZERO_OK)
        return st;
    if ((st = zero_gather_params(L, unit, unit + 1, w_shards, L->parts, w_full, stream)) != ZERO_OK)
        return st;
    // Y = X W: a(i, k) = X[i][k], b(j, k) = W[k][j]
    return zero_gemm_bf16(batch, d.out, d.in, x, d.in, ZERO_K_INNER, w_full, d.out, ZERO_K_OUTER,
                          y, d.out, y_dtype, stream);
}

zero_status zero_fsdp_linear_backward(const zero_layout *L, int32_t unit,
                                      const uint16_t *const *w_shards, int64_t batch,
                                      const uint16_t *x, const uint16_t *dy, uint16_t *w_full,
                                      void *dx, int32_t dx_dtype, float *dw_full, void *stream)
{
    Dims d;
    zero_status st = layer_dims(L, unit, &d);
    if (st != ZERO_OK)
        return st;
    if (!w_shards || !x || !dy || !w_full || !dx || !dw_full || batch < 0)
        return zs::fail(ZERO_ERR_INVALID_ARG, "every buffer and batch >= 0 are required");
    if ((st = check_shards(L, w_shards)) != ZERO_OK)
        return st;
    if (d.in % 8 || d.out % 8 || batch % 8)
        return zs::fail(ZERO_ERR_UNSUPPORTED, "in_features, out_features and batch must be "
                        "multiples of 8");
    // every check before the first launch: both GEMMs' too
    if ((st = zs::gemm_check(batch, d.in, d.out, dy, d.out, ZERO_K_INNER, w_full, d.out,
                             ZERO_K_INNER, dx, d.in, dx_dtype)) != ZERO_OK ||
        (st = zs::gemm_check(d.in, d.out, batch, x, d.in, ZERO_K_OUTER, dy, d.out, ZERO_K_OUTER,
                             dw_full, d.out, ZERO_FP32)) != ZERO_OK)
        return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    // re-gather W (FSDP frees it after forward)
    if ((st = zero_gather_params(L, unit, unit + 1, w_shards, L->parts, w_full, stream)) != ZERO_OK)
        return st;
    // dX = dY W^T: a(i, k) = dY[i][k], b(j, k) = W[j][k]
    if ((st = zero_gemm_bf16(batch, d.in, d.out, dy, d.out, ZERO_K_INNER, w_full, d.out,
                             ZERO_K_INNER, dx, d.in, dx_dtype, stream)) != ZERO_OK)
        return st;
    // dW = X^T dY, fp32, full shape: a(i, k) = X[k][i], b(j, k) = dY[k][j]
    if ((st = zero_gemm_bf16(d.in, d.out, batch, x, d.in, ZERO_K_OUTER, dy, d.out, ZERO_K_OUTER,
                             dw_full, d.out, ZERO_FP32, stream)) != ZERO_OK)
        return st;
    // padding rows of the row-sharded layout hold zero gradient
    return zs::zero_rows_fill(dw_full, d.out, d.in, d.in_pad, d.out, s);
}

// The layer with its epilogue: the checks of every step first, then the
// all-gather and one product.
zero_status zero_fsdp_linear_act_forward(const zero_layout *L, int32_t unit,
                                         const uint16_t *const *w_shards, int64_t batch,
                                         const uint16_t *x, uint16_t *w_full,
                                         const zero_epilogue *epilogue, void *y, int32_t y_dtype,
                                         void *stream)
{
    Dims d;
    zero_status st = layer_dims(L, unit, &d);
    if (st != ZERO_OK)
        return st;
    if (!w_shards || !w_full || batch < 0 || (batch > 0 && (!x || !y)))
        return zs::fail(ZERO_ERR_INVALID_ARG, "w_shards, x, w_full, y and batch >= 0 are "
                        "required");
    if ((st = check_shards(L, w_shards)) != ZERO_OK)
        return st;
    if (d.in % 8 || d.out % 8)
        return zs::fail(ZERO_ERR_UNSUPPORTED, "in_features and out_features must be "
                        "multiples of 8");
    if ((st = zs::gemm_check(batch, d.out, d.in, x, d.in, ZERO_K_INNER, w_full, d.out,
                             ZERO_K_OUTER, y, d.out, y_dtype)) != ZERO_OK ||
        (st = zs::epilogue_check(batch, d.out, x, w_full, y, d.out, y_dtype, epilogue,
                                 nullptr)) != ZERO_OK ||
        (batch > 0 &&
         (st = check_gathered(L, w_shards, w_full, x, nullptr, epilogue, y)) != ZERO_OK))
        return st;
    if ((st = zero_gather_params(L, unit, unit + 1, w_shards, L->parts, w_full, stream)) != ZERO_OK)
        return st;
    return zs::epilogue_gemm_run(batch, d.out, d.in, x, d.in, ZERO_K_INNER, w_full, d.out,
                                 ZERO_K_OUTER, y, d.out, y_dtype, epilogue,
                                 static_cast<hipStream_t>(stream));
}

zero_status zero_fsdp_linear_act_backward(const zero_layout *L, int32_t unit,
                                          const uint16_t *const *w_shards, int64_t batch,
                                          const zero_saved *x, int32_t act,
                                          const zero_saved *preact, const uint16_t *dy,
                                          uint16_t *w_full, uint16_t *dz, void *dx,
                                          int32_t dx_dtype, float *dw_full, float *dbias,
                                          float *workspace, int64_t n_workspace, void *stream)
{
    Dims d;
    zero_status st = layer_dims(L, unit, &d);
    if (st != ZERO_OK)
        return st;
    if (!w_shards || !x || !w_full || !dw_full || batch < 0 || (batch > 0 && (!dy || !dx)))
        return zs::fail(ZERO_ERR_INVALID_ARG, "w_shards, x, dy, w_full, dx, dw_full and batch >= 0 "
                        "are required");
    if ((st = check_shards(L, w_shards)) != ZERO_OK)
        return st;
    if (d.in % 8 || d.out % 8)
        return zs::fail(ZERO_ERR_UNSUPPORTED, "in_features and out_features must be "
                        "multiples of 8");
    if (act != ZERO_ACT_NONE && !dz && batch > 0)
        return zs::fail(ZERO_ERR_INVALID_ARG, "dz is required for an activation");
    // Without an activation dz is dy itself.
    const uint16_t *g = act == ZERO_ACT_NONE ? dy : dz;
    const bool elementwise = act != ZERO_ACT_NONE || dbias;
    if (elementwise &&
        (st = zs::act_backward_check(batch, d.out, dy, d.out, ZERO_BF16, act, preact,
                                     act == ZERO_ACT_NONE ? nullptr : dz, d.out, dbias, workspace,
                                     n_workspace)) != ZERO_OK)
        return st;
    if ((st = zs::gemm_check(batch, d.in, d.out, g, d.out, ZERO_K_INNER, w_full, d.out,
                             ZERO_K_INNER, dx, d.in, dx_dtype)) != ZERO_OK ||
        (st = zs::gemm_saved_check(d.in, d.out, batch, x, g, d.out, dw_full, d.out,
                                   ZERO_FP32)) != ZERO_OK)
        return st;
    // In the order of the work: w_full is gathered over nothing that is read
    // later; dz, dbias and the workspace leave x and w_full to the products (and
    // dbias is a result), dx leaves x, dz and dbias, dW the results.
    const bool kept = act != ZERO_ACT_NONE;
    const void *z = kept ? data_of(preact) : nullptr, *z_scales = kept ? scales_of(preact) : nullptr;
    const void *x8 = scales_of(x);
    const void *w = dbias && zero_act_backward_workspace(batch, d.out) > 0 ? workspace : nullptr;
    if (batch > 0 &&
        (is_one_of(w_full, {x->data, x8, dy, z, z_scales, g, dx, dbias, w}) ||
         (kept && is_one_of(dz, {x->data, x8})) || is_one_of(w, {x->data, x8}) ||
         is_one_of(dbias, {x->data, x8}) || is_one_of(dx, {x->data, x8, g, dbias}) ||
         is_one_of(dw_full, {x->data, x8, g, dx, dbias})))
        return zs::fail(ZERO_ERR_INVALID_ARG, "w_full, dz, dbias, the workspace, dx and dw_full must not lie "
                        "where x, w_full, dz or a result is still read or kept");
    if ((st = check_results(L, w_shards, {batch > 0 && kept ? dz : nullptr, batch > 0 ? dx : nullptr, dw_full,
                                          dbias, w})) != ZERO_OK)
        return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if ((st = zero_gather_params(L, unit, unit + 1, w_shards, L->parts, w_full, stream)) != ZERO_OK)
        return st;
    if (elementwise &&
        (st = zs::act_backward_run(batch, d.out, dy, d.out, ZERO_BF16, act, preact,
                                   act == ZERO_ACT_NONE ? nullptr : dz, d.out, dbias, workspace,
                                   s)) != ZERO_OK)
        return st;
    // dX = dZ W^T and dW = X^T dZ from the kept X, as in
    // zero_fsdp_linear_backward
    if ((st = zs::gemm_run(batch, d.in, d.out, g, d.out, ZERO_K_INNER, w_full, d.out, ZERO_K_INNER,
                           dx, d.in, dx_dtype, s)) != ZERO_OK)
        return st;
    if ((st = zs::gemm_saved_run(d.in, d.out, batch, x, g, d.out, dw_full, d.out, ZERO_FP32,
                                 s)) != ZERO_OK)
        return st;
    return zs::zero_rows_fill(dw_full, d.out, d.in, d.in_pad, d.out, s);
}

// The expert layer: unit `unit` holds the experts' in x out weights one after
// the other, so the unit has n_experts * in rows and its shards may cut
// through an expert; the gathered unit is the operand of the grouped product.
zero_status zero_fsdp_experts_forward(const zero_layout *L, int32_t unit, int32_t n_experts,
                                      const uint16_t *const *w_shards, const int64_t *offsets,
                                      int64_t rows, const uint16_t *x, uint16_t *w_full,
                                      const zero_epilogue *epilogue, void *y, int32_t y_dtype,
                                      void *stream)
{
    Dims d;
    zero_status st = expert_dims(L, unit, n_experts, &d);
    if (st != ZERO_OK)
        return st;
    if (!w_shards || !w_full || rows < 0 || (rows > 0 && (!x || !y)))
        return zs::fail(ZERO_ERR_INVALID_ARG, "w_shards, x, w_full, y and rows >= 0 are required");
    if ((st = check_shards(L, w_shards)) != ZERO_OK)
        return st;
    const int64_t stride = d.in * d.out;
    if ((st = zs::grouped_rows_check(n_experts, offsets, rows, d.out, d.in, x, d.in, w_full, d.out,
                                     ZERO_K_OUTER, stride, y, d.out, y_dtype, epilogue)) != ZERO_OK ||
        (rows > 0 &&
         (st = check_gathered(L, w_shards, w_full, x, offsets, epilogue, y)) != ZERO_OK))
        return st;
    if ((st = zero_gather_params(L, unit, unit + 1, w_shards, L->parts, w_full, stream)) != ZERO_OK)
        return st;
    return zs::grouped_rows_run(n_experts, offsets, rows, d.out, d.in, x, d.in, w_full, d.out, ZERO_K_OUTER,
                                stride, y, d.out, y_dtype, epilogue,
                                static_cast<hipStream_t>(stream));
}

zero_status zero_fsdp_experts_backward(const zero_layout *L, int32_t unit, int32_t n_experts,
                                       const uint16_t *const *w_shards, const int64_t *offsets,
                                       int64_t rows, const uint16_t *x, const uint16_t *dy,
                                       uint16_t *w_full, void *dx, int32_t dx_dtype,
                                       float *dw_full, void *stream)
{
    Dims d;
    zero_status st = expert_dims(L, unit, n_experts, &d);
    if (st != ZERO_OK)
        return st;
    if (!w_shards || !w_full || !dw_full || rows < 0 || (rows > 0 && (!x || !dy || !dx)))
        return zs::fail(ZERO_ERR_INVALID_ARG, "every buffer and rows >= 0 are required");
    if ((st = check_shards(L, w_shards)) != ZERO_OK)
        return st;
    const int64_t stride = d.in * d.out;
    if ((st = zs::grouped_rows_check(n_experts, offsets, rows, d.in, d.out, dy, d.out, w_full, d.out,
                                     ZERO_K_INNER, stride, dx, d.in, dx_dtype, nullptr)) != ZERO_OK ||
        (st = zs::grouped_depth_check(n_experts, offsets, rows, d.in, d.out, x, d.in, dy, d.out,
                                      dw_full, d.out, stride, ZERO_FP32)) != ZERO_OK)
        return st;
    if (rows > 0 && (is_one_of(dx, {x, dw_full}) || is_one_of(w_full, {x, dy, offsets})))
        return zs::fail(ZERO_ERR_INVALID_ARG, "dx must not lie where x is still read or dw_full is written, nor "
                        "w_full where x, dy or the offsets are still read");
    if ((st = check_results(L, w_shards, {rows > 0 ? dx : nullptr, dw_full})) != ZERO_OK)
        return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if ((st = zero_gather_params(L, unit, unit + 1, w_shards, L->parts, w_full, stream)) != ZERO_OK)
        return st;
    if ((st = zs::grouped_rows_run(n_experts, offsets, rows, d.in, d.out, dy, d.out, w_full, d.out,
                                   ZERO_K_INNER, stride, dx, d.in, dx_dtype, nullptr, s)) != ZERO_OK)
        return st;
    if ((st = zs::grouped_depth_run(n_experts, offsets, rows, d.in, d.out, x, d.in, dy, d.out, dw_full,
                                    d.out, stride, ZERO_FP32, s)) != ZERO_OK)
        return st;
    const int64_t total = d.in * n_experts;
    return zs::zero_rows_fill(dw_full, d.out, total, d.in_pad, d.out, s);
}

}  // extern "C"
