/*
 * zero_shard.h -- C ABI of the per-rank sharded mixed-precision optimizer
 * step for one AMD Instinct MI355X (gfx950) GPU.
 *
 * One data-parallel rank's step, seen from its own GPU, with the N ranks'
 * gradient buffers resident in this GPU's memory:
 *   reduce    the N ranks' gradients into this rank's 1/N slice, in fp32,
 *             divided by N -- the arithmetic of a reduce-scatter
 *             ("DP, ZeRO-1/2/3, FSDP" notes, concepts "reduce-scatter and
 *             all-gather"; "Data Parallel, ZeRO and FSDP", plain DDP);
 *   adam      Adam / AdamW on the slice's fp32 master, m and v (the 12 bytes
 *             per parameter that ZeRO shards; "DP, ZeRO-1/2/3, FSDP" notes,
 *             concepts "Model states" and "ZeRO-1 / 2 / 3"); the update
 *             equations are Kingma & Ba (2015) Algorithm 1, with
 *             Loshchilov & Hutter (2019) decoupled decay for AdamW;
 *   cast      the new master rounded to bf16 (round to nearest even) and
 *             stored at the rank's offsets of the flat parameter buffer;
 *   gather    the other ranks' bf16 slices packed into the full flat buffer
 *             -- the data movement of an all-gather.
 * Plus the DDP variant (no sharding: every replica averages and updates the
 * whole buffer) and the Megatron distributed-optimizer pieces (fp32 main
 * gradient accumulation; fp32 gradients reduced; "DP, ZeRO-1/2/3, FSDP"
 * notes, worked example, note under the Megatron row).
 *
 * LAYOUT (FSDP1-style flat parameter; "DP, ZeRO-1/2/3, FSDP" notes,
 * follow-up "FSDP2 vs FSDP1"): the parameters form units u = 0..U-1 of n_u
 * elements (a layer, or a gradient bucket).  Each unit is padded with zeros
 * at its tail to L_u = ceil(n_u / N) * N and the units are concatenated:
 *     F_u = sum_{j<u} L_j          (flat offset of unit u)
 *     s_u = L_u / N                (each rank's slice of unit u)
 *     R_u = sum_{j<u} s_j          (offset of unit u in a rank's shard)
 * Rank r owns flat elements [F_u + r*s_u, F_u + (r+1)*s_u) of every unit.
 * Under ZERO_DDP nothing is sharded: s_u = L_u = n_u and every rank "owns"
 * the whole buffer.
 *
 * RANGES AND INDEXING.  Every compute call covers a contiguous range of
 * units [unit_begin, unit_end) and every buffer pointer passed to it
 * addresses the first element of that range:
 *   ZERO_INDEX_FULL  buffer over the flat layout: element j of rank q's
 *                    slice of unit u is at (F_u - F_begin) + q*s_u + j;
 *   ZERO_INDEX_SHARD buffer over one rank's shard: element j of unit u is at
 *                    (R_u - R_begin) + j.
 * With unit_begin = 0 these are plain whole-buffer offsets; with a single
 * unit they address per-unit buffers (FSDP's gather / free per unit).
 * fp32 master, m and v are always shard-indexed: three such arrays, or, on a
 * layout made by zero_layout_chunk_state, one buffer over the whole shard
 * addressed from its start whatever the range.
 *
 * CONVENTIONS.
 *   - Lengths are element counts (int64_t).  Data pointers are DEVICE
 *     pointers owned by the caller; pointer ARRAYS (rank lists) and config
 *     structs are HOST memory, read during the call only.
 *   - `stream` is a hipStream_t (NULL = the null stream).  Every compute call
 *     only enqueues work on it and never synchronises.
 *   - Arguments are validated on the host before anything is launched; on
 *     any error nothing is launched and no buffer is touched.  Launch
 *     failures return ZERO_ERR_HIP.  zero_last_error() returns a text
 *     description of the last error on the calling thread.
 *   - The library allocates no device memory; a layout is host memory only
 *     and is immutable after init (safe to share between threads).
 *   - Every compute call only launches kernels (no memset, no copy, no
 *     allocation), so it may be captured into a HIP graph and replayed.
 *     zero_fsdp_sweep forks its gather stream from the step stream through
 *     events and joins it back before returning, so a capture of the step
 *     stream takes in both.  A graph keeps the argument values of its
 *     capture, the Adam step number included.
 *   - Calls that write disjoint buffers may run concurrently on different
 *     streams.  An fp32 buffer pointer must be 4-byte aligned and a bf16
 *     one 2-byte aligned; 16-byte aligned buffers with slice offsets that are
 *     multiples of 8 take the 128-bit vector path, others a scalar path with
 *     identical results.
 *   - At most ZERO_MAX_RANKS_PER_CALL rank buffers per reduce call.
 *   - Arithmetic: fp32, one IEEE-754 rounding per operation, no fused
 *     multiply-add; the N ranks are summed in ascending rank order from +0
 *     and the sum divided by N; results do not depend on the launch shape.
 */
#ifndef ZERO_SHARD_H
#define ZERO_SHARD_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define ZERO_MAX_RANKS_PER_CALL 64

typedef enum zero_status {
    ZERO_OK = 0,
    ZERO_ERR_INVALID_ARG = 1, /* null / out-of-range / inconsistent argument */
    ZERO_ERR_ALIGNMENT = 2,   /* pointer not aligned to its element size     */
    ZERO_ERR_OOM = 3,         /* host allocation failed                       */
    ZERO_ERR_HIP = 4,         /* a HIP runtime call or launch failed          */
    ZERO_ERR_UNSUPPORTED = 5  /* valid request outside this library's limits  */
} zero_status;

/* Who holds what ("DP, ZeRO-1/2/3, FSDP" notes, figure 1 and worked example;
   "Data Parallel, ZeRO and FSDP", ZeRO/FSDP table).  Only ZERO_DDP changes
   the layout (unsharded); the others record the caller's strategy. */
typedef enum zero_strategy {
    ZERO_DDP = 0,
    ZERO_STAGE1 = 1,
    ZERO_STAGE2 = 2,
    ZERO_STAGE3 = 3,
    ZERO_FSDP = 4,
    ZERO_MEGATRON_DO = 5
} zero_strategy;

typedef enum zero_dtype { ZERO_BF16 = 0, ZERO_FP32 = 1 } zero_dtype;

typedef enum zero_index { ZERO_INDEX_FULL = 0, ZERO_INDEX_SHARD = 1 } zero_index;

typedef struct zero_layout zero_layout;

/* The N ranks' gradient buffers for one call, all of one dtype (bf16 as raw
   uint16 bit patterns, or fp32).

   Chunked gradients (chunk = E > 0): the shard-indexed contributions to
   this rank's part of the call's range sit in one receive buffer R of
   ceil(S/E) rows, each row holding E elements of rank 0, then E of rank 1,
   ..., then E of rank N-1 (S = the range's shard length).  Rank q's
   gradient for element i of the range (counted from its first element, as
   for every shard-indexed buffer) is at R + (i / E) N E + q E + i % E, and
   ptrs[q] must be R + qE elements (ZERO_ERR_INVALID_ARG otherwise; at
   least one rank shard-indexed).  A full-indexed rank -- a rank's own
   main gradient, as in the Megatron distributed optimizer -- keeps its own
   buffer at ptrs[q]; its slot in R is never read.  A per-unit call
   therefore takes a per-unit receive buffer.
   The same bytes and sums as N separate buffers, read from one region
   instead of N: it is the receive buffer a rank would let its peers fill
   in a reduce-scatter.  On one MI355X the 7B / N = 8 fused step (state
   chunked either way) takes 0.956 x the time of eight separate buffers
   with E = 16384 (0.934-1.014 over six buffer placements; 2048-32768 all
   within 0.4 % of it).  E is a power of two in [ZERO_STATE_CHUNK_MIN,
   ZERO_STATE_CHUNK_MAX]. */
#define ZERO_GRAD_CHUNK_DEFAULT 16384 /* the measured best on MI355X */
typedef struct zero_grads {
    const void *const *ptrs; /* host array of n device pointers, rank order;
                                a NULL entry is an error (missing replica)  */
    const uint8_t *index;    /* host array of n zero_index values, or NULL
                                for all `index_all`                          */
    int32_t n;               /* must equal the layout's world_n             */
    int32_t dtype;           /* zero_dtype                                  */
    int32_t index_all;       /* zero_index used when `index` is NULL        */
    int32_t chunk;           /* 0: one buffer per rank; E: chunked (above)  */
} zero_grads;

/* Adam / AdamW hyper-parameters of one step.  The step scalars 1 - beta1,
   1 - beta2, 1 - beta1^t, 1 - beta2^t and 1 - lr*wd are evaluated in fp64
   from these fp32 values and rounded once to fp32. */
typedef struct zero_adam_cfg {
    float lr;
    float beta1;        /* in [0, 1) */
    float beta2;        /* in [0, 1) */
    float eps;          /* >= 0 */
    float weight_decay; /* >= 0; 0 disables both decay forms */
    int32_t decoupled;  /* 1: AdamW, p *= 1 - lr*wd; 0: L2, g += wd*p */
    int64_t step;       /* t >= 1, supplied by the caller every call */
} zero_adam_cfg;

/* ------------------------------------------------------------ layout -- */

/* Plan the layout of one rank: `n_units` units of unpadded sizes
   `unit_numel` (host array, each >= 0, at least one unit), `world_n` >= 1
   ranks, this rank `rank` in [0, world_n).  Host memory only; no HIP call.
   *out receives a layout to free with zero_shard_destroy.
   Source: "DP, ZeRO-1/2/3, FSDP" notes, concepts "ZeRO-1 / 2 / 3" (the
   model states are cut into N parts by data-parallel rank; each rank keeps
   and updates only its part) and "FSDP" (the model is split into units),
   and the follow-up "FSDP2 vs FSDP1" (FSDP1 flattens and concatenates a
   unit's parameters into one flat buffer and shards that); "Data Parallel,
   ZeRO and FSDP", section "ZeRO and FSDP".  The padding of each unit to a
   multiple of N is this layout's reading (the pages do not say how an
   uneven unit is cut). */
zero_status zero_shard_init(zero_layout **out, zero_strategy strategy,
                            int32_t world_n, int32_t rank, int32_t n_units,
                            const int64_t *unit_numel);

/* FSDP2-style per-parameter dim-0 sharding ("DP, ZeRO-1/2/3, FSDP" notes,
   follow-up "FSDP2 vs FSDP1": every parameter sharded on its own along dim
   0, so a rank holds whole rows and its sharded state dict needs no
   gather).  Unit u is a parameter of unit_rows[u] x unit_cols[u] elements
   (row-major; unit_cols >= 1, unit_rows >= 0).  It is cut into chunks of
   c_u = ceil(rows / N) rows (the torch.chunk rule): rank r holds rows
   [r c_u, min((r+1) c_u, rows)), padded with zero rows to c_u rows, so
   s_u = c_u * cols and L_u = N * s_u.  Offsets F_u, R_u and every other
   call work exactly as for zero_shard_init. */
zero_status zero_shard_init_rows(zero_layout **out, zero_strategy strategy,
                                 int32_t world_n, int32_t rank,
                                 int32_t n_units, const int64_t *unit_rows,
                                 const int64_t *unit_cols);

void zero_shard_destroy(zero_layout *layout);

/* Whole-layout sizes: padded flat length sum L_u, this rank's shard length
   sum s_u.  Any output pointer may be NULL. */
zero_status zero_layout_info(const zero_layout *layout, int64_t *flat_len,
                             int64_t *shard_len, int32_t *n_units,
                             int32_t *world_n, int32_t *rank,
                             int32_t *strategy);

/* Per-unit numbers (see LAYOUT): n_u, L_u, F_u, s_u, R_u and the rank's
   flat offset F_u + r*s_u.  Any output pointer may be NULL.  These are the
   offsets of the flat-buffer sharding that zero_shard_init plans (same
   source): where unit u sits in the flat buffer, where its slice sits in a
   rank's shard, and which flat elements this rank owns. */
zero_status zero_layout_query(const zero_layout *layout, int32_t unit,
                              int64_t *numel, int64_t *padded_len,
                              int64_t *flat_off, int64_t *shard_len,
                              int64_t *shard_off, int64_t *rank_flat_off);

/* The rows of unit u this rank really holds (the rest of its slice is
   padding): *cols (1 for element-granular layouts), *first_row and
   *row_count (0 when this rank's chunk lies past the end).  For an
   element-granular layout rows are elements.  Any output may be NULL. */
zero_status zero_layout_rows(const zero_layout *layout, int32_t unit,
                             int64_t *cols, int64_t *first_row,
                             int64_t *row_count);

/* Chunked optimizer state.  The pages fix what a rank keeps per parameter
   (fp32 master, m and v: "DP, ZeRO-1/2/3, FSDP" notes, concepts "Model
   states"), not where it lies in memory.  *out receives a copy of `layout`
   (free it with zero_shard_destroy) whose master, m and v live in ONE
   buffer, interleaved in chunks of E = `chunk` elements: shard element i of
   master is at state[(i / E) * 3E + i % E], of m at E further, of v at 2E
   further.  Every call that takes master, m and v on such a layout expects
   master = state, m = state + E, v = state + 2E, where `state` is the start
   of a buffer of zero_layout_state(...) floats covering the whole shard,
   whatever the call's unit range (else ZERO_ERR_INVALID_ARG); the kernels
   add the range's shard offset themselves.  Results are bit-identical to
   the three-array layout; only addresses change.  The fused step reads and
   writes each chunk's three parts next to each other instead of in three
   arrays gigabytes apart, which HBM serves faster: on one MI355X the
   7B / N = 8 step kernel takes 0.938 x the three-array time with
   E = 8192 (0.910-0.982 over six buffer placements).  chunk = 0 gives the
   three-array format back; otherwise `chunk` is a power of two in
   [ZERO_STATE_CHUNK_MIN, ZERO_STATE_CHUNK_MAX]. */
#define ZERO_STATE_CHUNK_MIN 4
#define ZERO_STATE_CHUNK_MAX 16777216
#define ZERO_STATE_CHUNK_DEFAULT 8192 /* the measured best on MI355X */
zero_status zero_layout_chunk_state(const zero_layout *layout, int64_t chunk,
                                    zero_layout **out);

/* The layout's state format: *chunk = 0 (three arrays of shard_len floats,
   *state_len = shard_len) or E (one buffer of *state_len =
   ceil(shard_len / E) * 3E floats).  Either output may be NULL. */
zero_status zero_layout_state(const zero_layout *layout, int64_t *chunk,
                              int64_t *state_len);

/* ------------------------------------------------------------ reduce -- */

/* Reduce-scatter arithmetic: for every element of this rank's slices of
   units [unit_begin, unit_end),
       out[i] = (G_0[i] + G_1[i] + ... + G_{N-1}[i]) / N      (fp32)
   with G_q indexed as grads->index says.  `out` is fp32, indexed as
   `out_index` says: ZERO_INDEX_SHARD for this rank's reduce-scatter result,
   ZERO_INDEX_FULL to write this rank's slices into a full flat buffer (the
   N ranks' calls together then form the all-reduce).
   If `sumsq_partials` is non-NULL it receives exactly
   zero_reduce_partials_count(...) fp64 partial sums of out[i]^2 (each square
   exact in fp64; one partial per 1024-element tile of a unit slice, summed
   in a fixed order), for the global-norm clip; `n_partials` is the capacity
   of that buffer.
   Source: "DP, ZeRO-1/2/3, FSDP" notes, concepts "reduce-scatter and
   all-gather" (a reduce-scatter sums the ranks' buffers and leaves each
   rank 1/N of the result; with the all-gather it makes an all-reduce);
   "Data Parallel, ZeRO and FSDP", section "Plain data parallel (DDP)"
   (after the all-reduce every replica holds the mean gradient) and section
   "ZeRO and FSDP" (gradients are reduce-scattered so that each GPU keeps
   its shard).  Summing in ascending rank order is this library's reading. */
zero_status zero_reduce_shard(const zero_layout *layout, int32_t unit_begin,
                              int32_t unit_end, const zero_grads *grads,
                              float *out, int32_t out_index,
                              double *sumsq_partials,
                              int64_t n_partials, void *stream);

/* Number of fp64 partials zero_reduce_shard writes for a range: one per
   1024-element tile of every unit slice in the range (a fixed function of
   the range, independent of the device and of the launch width). */
int64_t zero_reduce_partials_count(const zero_layout *layout,
                                   int32_t unit_begin, int32_t unit_end);

/* Global gradient-norm clip coefficient.  Not on the pages: the
   GPT-2-small workload with a global-norm clip at 1.0 names it, and the
   reading taken is PyTorch's clip_grad_norm_:
   norm = sqrt(sum of the n partials in fp64, in
   a fixed order for a given n: strided per-thread sums, then a fixed tree),
   *coef_out = min(1, fp32(max_norm / (norm + 1e-6))).
   `partials`, `coef_out` (one float) and `norm_out` (one double, may be
   NULL) are device pointers.  n >= 1, max_norm > 0. */
zero_status zero_clip_coef(const double *partials, int64_t n, float max_norm,
                           float *coef_out, double *norm_out, void *stream);

/* ------------------------------------------------ no allocation -- */

/* Capacity of the library's static device buffer of sum-of-squares partials
   (4 MiB of fp64 per GPU, held until the process ends). */
#define ZERO_NOALLOC_MAX_PARTIALS 524288

/* For callers that cannot allocate device memory: code under HIP graph
   capture, tight serving loops, harnesses that forbid hipMalloc.  The
   two-pass clipped step of one range -- zero_reduce_shard into `grad_out`
   (fp32, shard-indexed) with sum-of-squares partials, zero_clip_coef over
   those partials (max_norm > 0), then zero_adam_step from `grad_out` scaled
   by the coefficient -- with the partials and the coefficient kept in a
   static device array of the library instead of caller buffers.  Results
   are those of that three-call sequence, bit for bit.  The norm is the
   norm of this call's range: the whole buffer under ZERO_DDP, this rank's
   shard otherwise (a global norm over several ranks needs every rank's
   partials: use the three calls).  `norm_out` (device double, may be NULL)
   receives the norm.  The range may need at most ZERO_NOALLOC_MAX_PARTIALS
   partials (zero_reduce_partials_count; 536,870,912 elements per rank),
   else ZERO_ERR_UNSUPPORTED.  The call allocates nothing and calls no
   allocating routine; every argument is checked on the host before the
   first HIP call.  Calls on one GPU share its array, so calls that overlap
   in time on one GPU (other streams, other host threads) race; calls in
   one stream order are safe, each overwriting what it uses before reading
   it. */
zero_status zero_adam_step_clip_noalloc(const zero_layout *layout, int32_t unit_begin,
                                        int32_t unit_end, const zero_adam_cfg *cfg,
                                        float max_norm, const zero_grads *grads,
                                        float *grad_out, float *master, float *m, float *v,
                                        uint16_t *param_out, int32_t param_index,
                                        double *norm_out, void *stream);

/* --------------------------------------------------------- Adam step -- */

/* Adam / AdamW on this rank's slices of units [unit_begin, unit_end), then
   bf16 rounding of the new master into `param_out`.
   Source: "DP, ZeRO-1/2/3, FSDP" notes, concepts "Model states" (bf16
   parameter and gradient, fp32 master, m and v: 12 of the 16 bytes per
   parameter) and "ZeRO-1 / 2 / 3" (each rank updates only its part); the
   update itself is Kingma & Ba (2015) Algorithm 1 and, for AdamW,
   Loshchilov & Hutter (2019), as the pages leave it to the optimizer.
   Gradient source, exactly one of:
     grad_fp32 != NULL: fp32 averaged gradient, indexed as `grad_index`
                        says: ZERO_INDEX_SHARD for a reduce-scatter result
                        (zero_reduce_shard on this layout), ZERO_INDEX_FULL
                        for an all-reduce result over this layout's whole
                        flat buffer (zero_reduce_shard of every rank's
                        layout with out_index = ZERO_INDEX_FULL -- ZeRO-1
                        implemented with all-reduce, "DP, ZeRO-1/2/3, FSDP"
                        notes, follow-up on the ZeRO-1 / ZeRO-2
                        communication gap); multiplied by *clip_coef (a
                        device float; NULL means 1);
     grads != NULL:     fused path -- the N ranks' buffers are reduced
                        (as zero_reduce_shard) in the same pass, so each
                        byte crosses HBM once.  clip_coef must be NULL.
   master, m, v: shard-indexed fp32, updated in place.
   param_out: bf16 (uint16) written at the rank's offsets; `param_index`
   says whether it is the full flat buffer (ZERO_INDEX_FULL: elements of
   the other ranks are not touched) or the rank's own shard buffer
   (ZERO_INDEX_SHARD, ZeRO-3 / FSDP). */
zero_status zero_adam_step(const zero_layout *layout, int32_t unit_begin,
                           int32_t unit_end, const zero_adam_cfg *cfg,
                           const float *grad_fp32, int32_t grad_index,
                           const float *clip_coef,
                           const zero_grads *grads, float *master, float *m,
                           float *v, uint16_t *param_out, int32_t param_index,
                           void *stream);

/* Step scalars read on the device, for graph replay.  A captured graph keeps
   the arguments of its capture, so zero_adam_step replayed from a graph
   would repeat one step number (and one learning rate).
   zero_adam_step_table instead reads the step's scalars when its kernels
   run, from entry (*step_counter - 1) of a table that the caller fills once
   on the host with zero_adam_table_fill and copies to the device.
   zero_step_advance increments the counter on the device.  A graph of
   [zero_adam_step_table, ..., zero_step_advance] then replays as steps 1,
   2, 3, ... with the arithmetic of zero_adam_step, bit for bit.
   The entry is the set of fp32 scalars of one step, each evaluated in fp64
   from that step's configuration and rounded once (as zero_adam_step). */
typedef struct zero_adam_table_entry {
    float lr, beta1, beta2, eps, weight_decay;
    float one_minus_beta1, one_minus_beta2;
    float bias1, bias2;  /* 1 - beta1^t, 1 - beta2^t of the entry's step t */
    float decay;         /* 1 - lr * weight_decay */
    int32_t has_decay;   /* weight_decay != 0 */
    int32_t decoupled;
} zero_adam_table_entry;

/* host_out[k] = the step scalars of cfgs[k], k < n (host arrays; each cfg
   validated as in zero_adam_step).  cfgs[k].step is the t of entry k,
   normally k + 1; lr may change from entry to entry (a schedule). */
zero_status zero_adam_table_fill(const zero_adam_cfg *cfgs, int64_t n,
                                 zero_adam_table_entry *host_out);

/* zero_adam_step with the scalars of table[*step_counter - 1].  `table` is
   a device array of n_entries >= 1 entries (4-byte aligned), `step_counter`
   a device int64 (8-byte aligned), both read when the kernels run; a
   counter outside [1, n_entries] leaves every buffer untouched.  The other
   arguments, and the host-side errors, are those of zero_adam_step. */
zero_status zero_adam_step_table(const zero_layout *layout, int32_t unit_begin,
                                 int32_t unit_end, const zero_adam_table_entry *table,
                                 int64_t n_entries, const int64_t *step_counter,
                                 const float *grad_fp32, int32_t grad_index,
                                 const float *clip_coef, const zero_grads *grads,
                                 float *master, float *m, float *v, uint16_t *param_out,
                                 int32_t param_index, void *stream);

/* *step_counter += 1 on the device, in stream order (device int64,
   8-byte aligned). */
zero_status zero_step_advance(int64_t *step_counter, void *stream);

/* ------------------------------------------------------------ gather -- */

/* All-gather data movement (source: "DP, ZeRO-1/2/3, FSDP" notes, concepts
   "reduce-scatter and all-gather": an all-gather puts the ranks' 1/N
   slices back together into the whole; "Data Parallel, ZeRO and FSDP",
   section "ZeRO and FSDP": a layer's parameter shards are all-gathered
   before it runs): for every rank q < n with shards[q] != NULL
   and every element j of rank q's slice of unit u in the range,
       param_full[(F_u - F_begin) + q*s_u + j] = shards[q][(R_u - R_begin) + j]
   Bit copies.  `shards` is a host array of n = world_n device pointers
   (NULL entries are skipped -- typically this rank's own, already written by
   zero_adam_step); param_full is the full flat bf16 buffer of the range. */
zero_status zero_gather_params(const zero_layout *layout, int32_t unit_begin,
                               int32_t unit_end, const uint16_t *const *shards,
                               int32_t n, uint16_t *param_full, void *stream);

/* ------------------------------------------------------ FSDP sweep -- */

/* One unit's buffers for zero_fsdp_sweep. */
typedef struct zero_unit_io {
    const void *const *rank_grads;      /* host array of world_n device pointers:
                                           this unit's rank gradients, each
                                           indexed over this rank's slice of the
                                           unit (s_u elements, unit-local); or,
                                           with grad_chunk > 0, the pointers of
                                           this unit's chunked receive buffer
                                           (zero_grads.chunk)                  */
    const uint16_t *const *peer_shards; /* host array of world_n device pointers
                                           (s_u bf16 each) gathered into the
                                           unit buffer; NULL entries skipped,
                                           this rank's own entry must be NULL  */
    uint16_t *unit_full;                /* device, L_u bf16: the unit's full
                                           flat parameters                     */
} zero_unit_io;

/* The FSDP per-unit sweep as a two-stream pipeline ("DP, ZeRO-1/2/3, FSDP"
   notes, follow-up on how FSDP hides communication: the all-gather runs on
   its own stream, the next unit's gather is prefetched, and
   limit_all_gathers bounds how many gathered units exist at once).
   For every unit u in [unit_begin, unit_end), in order:
     on step_stream:   the fused reduce of io[u].rank_grads (grad_dtype) +
                       Adam + bf16 of this rank's slice into io[u].unit_full
                       (zero_adam_step on the single unit; master, m and v
                       are shard-indexed from unit_begin, as everywhere, or
                       a chunked state from its start);
     on gather_stream: after that step, zero_gather_params of
                       io[u].peer_shards into io[u].unit_full (an all-gather
                       carries every rank's updated shard, so it follows the
                       step of its unit).
   max_inflight caps the pipeline: the step of unit u waits until the
   gather of unit u - max_inflight has finished.  1 makes the sweep
   sequential, 2 double-buffers (the step of unit u+1 overlaps the gather of
   unit u), 0 means no cap.  When the call's work completes on step_stream,
   every gather has completed too (step_stream waits for the last one).
   gather_stream may equal step_stream (sequential).  Results are identical
   to per-unit zero_adam_step + zero_gather_params calls.  Host-side errors
   launch nothing; a HIP error part-way returns ZERO_ERR_HIP with the units
   before it enqueued.  `io` is a host array of (unit_end - unit_begin)
   entries.  grad_chunk = 0 takes each unit's rank gradients as world_n
   buffers; E > 0 as one chunked receive buffer per unit, as
   zero_grads.chunk describes, checked for every unit before anything is
   launched. */
zero_status zero_fsdp_sweep(const zero_layout *layout, int32_t unit_begin,
                            int32_t unit_end, const zero_adam_cfg *cfg,
                            int32_t grad_dtype, int32_t grad_chunk,
                            const zero_unit_io *io,
                            float *master, float *m, float *v,
                            int32_t max_inflight, void *step_stream,
                            void *gather_stream);

/* zero_fsdp_sweep with each unit's step as zero_adam_step_table (scalars of
   table[*step_counter - 1], read on the device), then *step_counter += 1 on
   step_stream after the last unit's step: a graph captured from one call
   replays as the sweeps of steps 1, 2, 3, ... .  Arguments and errors
   otherwise as zero_fsdp_sweep and zero_adam_step_table. */
zero_status zero_fsdp_sweep_table(const zero_layout *layout, int32_t unit_begin,
                                  int32_t unit_end, const zero_adam_table_entry *table,
                                  int64_t n_entries, int64_t *step_counter,
                                  int32_t grad_dtype, int32_t grad_chunk,
                                  const zero_unit_io *io,
                                  float *master, float *m, float *v,
                                  int32_t max_inflight, void *step_stream,
                                  void *gather_stream);

/* ------------------------------------------------------- accumulation -- */

/* Megatron-style fp32 main-gradient accumulation of one micro-batch:
   main_grad[i] = main_grad[i] + float(micro_bf16[i]) for i < n.
   Source: "DP, ZeRO-1/2/3, FSDP" notes, worked example "7B, N = 8", the
   note under the Megatron distributed-optimizer row (the gradient is kept
   and accumulated in fp32: 4 bytes per parameter, replicated); the bf16
   micro-batch gradient is this library's reading (the model is bf16). */
zero_status zero_grad_accumulate(float *main_grad, const uint16_t *micro_bf16,
                                 int64_t n, void *stream);

/* ---------------------------------------------- rate calibration -- */

/* HBM rate of the fused step's memory traffic without its arithmetic, for
   measuring the step kernel against the ceiling of its own access pattern
   (a measurement aid, not part of the optimizer step).  Over elements
   i < n, with the launch shape, tile walk and per-lane element ownership of
   zero_adam_step's fused kernel, and every buffer indexed from 0:
     ZERO_MIX_STEP_STREAMS  reads the n_ranks bf16 grads[q][i] and master[i],
                            m[i], v[i]; writes master[i] + s, m[i] + s and
                            v[i] + s (s = the fp32 sum of the rank values) and
                            param[i] = the upper 16 bits of the new master[i];
     ZERO_MIX_READS         the same reads, nothing written;
     ZERO_MIX_WRITES        the same writes, nothing read (master, m, v and
                            param receive values derived from i).
   Per element the step streams are 2*n_ranks + 12 bytes read and 14 bytes
   written, as in the fused step.  `grads` is a host array of n_ranks device
   pointers; 1 <= n_ranks <= ZERO_MAX_RANKS_PER_CALL; n must be a multiple of
   4 and every buffer 16-byte aligned (ZERO_ERR_INVALID_ARG /
   ZERO_ERR_ALIGNMENT otherwise, nothing launched).  `state_chunk` = 0 takes
   master, m and v as three arrays; a power of two E in
   [ZERO_STATE_CHUNK_MIN, ZERO_STATE_CHUNK_MAX] takes them in the chunked
   format of zero_layout_chunk_state (m = master + E, v = master + 2E), so
   the calibration covers the same addresses as a chunked-state step.
   Likewise `grad_chunk` = 0 takes n_ranks separate gradient buffers, and a
   power of two E in the same bounds takes them chunked as zero_grads.chunk
   describes (grads[q] = grads[0] + qE; element i of rank q at
   grads[q] + (i / E) n_ranks E + i % E). */
typedef enum {
    ZERO_MIX_STEP_STREAMS = 0,
    ZERO_MIX_READS = 1,
    ZERO_MIX_WRITES = 2
} zero_mix_kind;

zero_status zero_stream_mix(int32_t kind, const uint16_t *const *grads, int32_t n_ranks,
                            float *master, float *m, float *v, uint16_t *param, int64_t n,
                            int64_t state_chunk, int64_t grad_chunk, void *stream);

/* ----------------------------------------------- FSDP linear layer -- */

/* How a GEMM operand is stored.  K_INNER: A as M x K, B as N x K (row-major,
   K contiguous).  K_OUTER: A as K x M, B as K x N (row-major, M or N
   contiguous). */
typedef enum {
    ZERO_K_INNER = 0,
    ZERO_K_OUTER = 1
} zero_operand_order;

/* C[i][j] = sum_{k < K} a(i, k) * b(j, k) for i < M, j < N on the MFMA
   units, where a(i, k) = A[i * lda + k] (K_INNER) or A[k * lda + i]
   (K_OUTER), and b(j, k) = B[j * ldb + k] (K_INNER) or B[k * ldb + j]
   (K_OUTER).  So with B K_OUTER this is C = A B, with both K_INNER
   C = A B^T, with both K_OUTER C = A^T B.  A and B are bf16 bits; C is
   row-major with leading dimension ldc, fp32 (c_dtype ZERO_FP32) or bf16
   rounded to nearest even (ZERO_BF16).  Accumulation is fp32 in the
   kernel's own order (error within the usual gamma_K bound of fp32 dot
   products).  Needs K, lda and ldb multiples of 8, M (N) a multiple of 8
   when A (B) is K_OUTER, lda >= K or M and ldb >= K or N by order,
   ldc >= N, and 16-byte aligned A and B.  Operands are read through 32-bit
   buffer offsets, so a K_INNER operand's leading dimension must be at most
   2^22 = 4,194,304 elements and a K_OUTER one's at most 2^25 = 33,554,432.
   C may span at most 4,194,303 tiles of 256 x 256 (the launch, up to two
   512-thread blocks per tile, stays below 2^32 work-items).
   ZERO_ERR_UNSUPPORTED or ZERO_ERR_ALIGNMENT otherwise, with nothing
   launched.  M = 0 or N = 0 is
   a no-op; K = 0 writes zeros.  All pointers are device memory owned by the
   caller. */
zero_status zero_gemm_bf16(int64_t M, int64_t N, int64_t K, const uint16_t *A,
                           int64_t lda, int32_t a_order, const uint16_t *B,
                           int64_t ldb, int32_t b_order, void *C, int64_t ldc,
                           int32_t c_dtype, void *stream);

/* zero_gemm_bf16 with both operands K_INNER: C = A B^T. */
zero_status zero_gemm_bf16_nt(int64_t M, int64_t N, int64_t K, const uint16_t *A,
                              int64_t lda, const uint16_t *B, int64_t ldb,
                              void *C, int64_t ldc, int32_t c_dtype,
                              void *stream);

/* dst[c * ldd + r] = src[r * lds + c] for r < rows, c < cols (bf16 bits). */
zero_status zero_transpose_bf16(int64_t rows, int64_t cols, const uint16_t *src,
                                int64_t lds, uint16_t *dst, int64_t ldd,
                                void *stream);

/* A hand-written FSDP linear layer ("DP, ZeRO-1/2/3, FSDP" notes, follow-up
   on writing one FSDP linear layer: each rank stores 1/N of the rows of W;
   forward all-gathers W and computes X W; backward all-gathers W again,
   computes dX and the full-shape dW locally, and reduce-scatters dW into
   each rank's rows).  W is unit `unit` of a row layout
   (zero_shard_init_rows): rows = in_features (in), cols = out_features
   (out), so rank r's W shard is its c_u x out rows.
   forward:  w_full = all-gather(w_shards) (device, L_u bf16 workspace);
             y = x W (x: batch x in bf16; y: batch x out, y_dtype).
   backward: w_full = all-gather(w_shards) again; dx = dy W^T (dy: batch x
             out bf16; dx: batch x in, dx_dtype); dw_full = x^T dy (fp32,
             the padded unit: in rows then zeroed padding rows, L_u
             elements).  The reduce-scatter of the N ranks' dw_full is
             zero_reduce_shard (fp32 grads, ZERO_INDEX_FULL) on this unit,
             and zero_adam_step(grad_fp32 = its output) steps the shard.
   Every GEMM reads its operands in place (zero_gemm_bf16 with K_OUTER
   operands), so no transposed copies are made.
   `w_shards` is a host array of world_n device pointers (s_u bf16 each, this
   rank's own included).  in and out must be multiples of 8, and batch too
   for the backward; x, dy, w_full and the shards 16-byte aligned. */
zero_status zero_fsdp_linear_forward(const zero_layout *layout, int32_t unit,
                                     const uint16_t *const *w_shards,
                                     int64_t batch, const uint16_t *x,
                                     uint16_t *w_full, void *y, int32_t y_dtype,
                                     void *stream);

zero_status zero_fsdp_linear_backward(const zero_layout *layout, int32_t unit,
                                      const uint16_t *const *w_shards,
                                      int64_t batch, const uint16_t *x,
                                      const uint16_t *dy, uint16_t *w_full,
                                      void *dx, int32_t dx_dtype,
                                      float *dw_full, void *stream);

/* ------------------------------------------------ layer operators -- */

/* What a linear layer does around its product, and what it keeps for its
   backward pass.  The pages leave the layer's inside to the model; they
   count the bytes a rank holds ("DP, ZeRO-1/2/3, FSDP" notes, concepts
   "Model states", which sets activations apart from the 16 bytes per
   parameter), and these calls are about the other part: fewer passes over
   the activations, and half the bytes of those kept.

   An activation, z -> act(z), in fp32: RELU max(z, 0); GELU z Phi(z);
   GELU_TANH z sigmoid(2 sqrt(2/pi) (z + 0.044715 z^3)); SILU z sigmoid(z).
   Infinities take their limits (act(-inf) = 0 for all but NONE), NaN stays
   NaN. */
typedef enum zero_activation {
    ZERO_ACT_NONE = 0,
    ZERO_ACT_RELU = 1,
    ZERO_ACT_GELU = 2,
    ZERO_ACT_GELU_TANH = 3,
    ZERO_ACT_SILU = 4
} zero_activation;

/* In all of these calls a matrix without rows (or a product's operand with
   K = 0) is never read, and its address may be NULL. */

/* A rows x cols activation matrix kept for the backward pass.
     ZERO_SAVED_BF16  data: rows x cols bf16, leading dimension ld.
     ZERO_SAVED_E4M3  data: rows x cols e4m3 codes of one byte, leading
                      dimension ld (a multiple of 16, data 16-byte aligned);
                      scales: ceil(rows / 32) x cols bytes, leading dimension
                      ld_scales.  One byte b serves the 32 rows (tokens)
                      32 i .. 32 i + 31 of one column (feature): the values
                      are code * 2^(b - 127), each exact in bf16.  b - 127 is
                      the least e in [-117, 120] for which the block's
                      largest finite magnitude is at most 448 * 2^e, and the
                      code is x / 2^e rounded to nearest even, |x| first
                      bounded by 240 * 2^120.  NaN and infinities become NaN
                      and do not count for e.
   Blocks run along tokens because dW = X^T dZ contracts over tokens, and so
   that a feature with large values costs its neighbours no precision. */
typedef enum zero_saved_format { ZERO_SAVED_BF16 = 0, ZERO_SAVED_E4M3 = 1 } zero_saved_format;

typedef struct zero_saved {
    void *data;
    int64_t ld;
    uint8_t *scales;   /* E4M3 only */
    int64_t ld_scales; /* E4M3 only */
    int32_t format;
} zero_saved;

/* *out = x (rows x cols, bf16 or fp32, leading dimension ldx) in 8 bits
   (E4M3 only).  Bytes past column cols of a row are not written.  The matrix,
   the codes and the scales need memory each, here and in zero_saved_read; an
   address given twice is refused. */
zero_status zero_saved_write(int64_t rows, int64_t cols, const void *x, int64_t ldx,
                             int32_t x_dtype, const zero_saved *out, void *stream);

/* out = the values *in stands for (E4M3 only; bf16 and fp32 both exact). */
zero_status zero_saved_read(int64_t rows, int64_t cols, const zero_saved *in, void *out,
                            int64_t ldo, int32_t out_dtype, void *stream);

/* The epilogue of an M x N product: with z = A B + bias,
       C = act(z) + residual,
   in fp32, C rounded once to its type.  NULL members are left out.
     bias      N values, bf16 or fp32;
     residual  M x N, bf16 or fp32, leading dimension ldr; it may be C itself
               (same type and leading dimension), else it must not overlap C;
     preact    receives z, in either format (E4M3: coded from the fp32 z);
     output    receives C in 8 bits (E4M3), coded from C as stored: the same
               bytes that zero_saved_write of C would give.
   What a call writes (C, preact, output, with their scales) needs memory apart
   from everything else that the call uses, the residual in place excepted; an
   address given twice is refused.  That holds for the scales and the offsets
   of the products below, too. */
typedef struct zero_epilogue {
    const void *bias;
    const void *residual;
    int64_t ldr;
    const zero_saved *preact;
    const zero_saved *output;
    int32_t bias_dtype;
    int32_t residual_dtype;
    int32_t act;
} zero_epilogue;

/* zero_gemm_bf16 with an epilogue (NULL: none).  Limits and errors as there,
   and the epilogue's matrices checked like C.  K = 0 gives z = bias. */
zero_status zero_gemm_bf16_epilogue(int64_t M, int64_t N, int64_t K, const uint16_t *A,
                                    int64_t lda, int32_t a_order, const uint16_t *B,
                                    int64_t ldb, int32_t b_order, void *C, int64_t ldc,
                                    int32_t c_dtype, const zero_epilogue *epilogue,
                                    void *stream);

/* The gradient of that epilogue:
       dz[i][j]  = dy[i][j] * act'(preact[i][j])     (bf16)
       dbias[j]  = sum over i of dz[i][j]            (fp32, of the unrounded
                                                      products; NULL: left out)
   The residual's gradient is dy itself.  dy is bf16 or fp32; dz may be dy or
   a bf16 preact (bf16, same leading dimension).  For ZERO_ACT_NONE preact is
   not read and dz may be NULL (dbias alone).  relu'(0) = 0; act'(NaN) is NaN.
   The sum runs in a fixed order, so dbias has the same bits every time; it needs
   `workspace` of zero_act_backward_workspace(rows, cols) floats (at most
   64 cols; 0 up to 128 rows, and the workspace may then be NULL), used
   until the call's work has run: calls that overlap in time, and captured
   graphs that do, need one each.  But for dz in place, one address for two
   things is refused.  rows = 0 writes zeros to dbias. */
zero_status zero_act_backward(int64_t rows, int64_t cols, const void *dy, int64_t ldy,
                              int32_t dy_dtype, int32_t act, const zero_saved *preact,
                              uint16_t *dz, int64_t ldz, float *dbias, float *workspace,
                              int64_t n_workspace, void *stream);
int64_t zero_act_backward_workspace(int64_t rows, int64_t cols);

/* C[i][j] = sum_{k < K} A[k][i] B[k][j] with A (K x M) kept in either format
   and B K x N bf16: a layer's dW = X^T dZ from the kept X, read in place.
   fp32 accumulation, C fp32 or bf16.  K is any number; M, N and the leading
   dimensions of A and B multiples of 8 (codes: 16; the scales' rows 4-byte
   aligned), at most 2^25; A and B 16-byte aligned.  K = 0 writes zeros. */
zero_status zero_gemm_saved_bf16(int64_t M, int64_t N, int64_t K, const zero_saved *A,
                                 const uint16_t *B, int64_t ldb, void *C, int64_t ldc,
                                 int32_t c_dtype, void *stream);

/* Products grouped by expert.  The rows of A are sorted by group: group e has
   the rows offsets[e] .. offsets[e + 1] - 1, where `offsets` is a DEVICE array
   of n_groups + 1 int64 (8-byte aligned) read when the kernels run -- a
   router's counts never come to the host, and a captured call takes new
   sizes at every replay.  Groups may be empty.  Offsets are clamped to
   [0, rows] and a decreasing pair to an empty group, so nothing outside the
   buffers is touched whatever the array holds; what such an array computes
   is unspecified.

   rows:   C[r] = epilogue(A[r] B_e), r in group e, with A rows x K bf16 and
           B_e = B + e * stride_b (elements, a multiple of 8), N and K and the
           orders as zero_gemm_bf16 has them (A K_INNER).  Rows in no group
           are left as they were, in C and in the kept pre-activation.  The
           epilogue has no bias and keeps nothing in 8 bits (a group does not
           begin at a multiple of 32 rows): ZERO_ERR_UNSUPPORTED.
   depth:  C_e[i][j] = sum over r in group e of A[r][i] B[r][j], C_e = C +
           e * stride_c (elements); an empty group's C_e is zeros.  A is
           rows x M, B rows x N, both bf16; any row count. */
zero_status zero_gemm_grouped_rows_bf16(int32_t n_groups, const int64_t *offsets, int64_t rows,
                                        int64_t N, int64_t K, const uint16_t *A, int64_t lda,
                                        const uint16_t *B, int64_t ldb, int32_t b_order,
                                        int64_t stride_b, void *C, int64_t ldc, int32_t c_dtype,
                                        const zero_epilogue *epilogue, void *stream);
zero_status zero_gemm_grouped_depth_bf16(int32_t n_groups, const int64_t *offsets, int64_t rows,
                                         int64_t M, int64_t N, const uint16_t *A, int64_t lda,
                                         const uint16_t *B, int64_t ldb, void *C, int64_t ldc,
                                         int64_t stride_c, int32_t c_dtype, void *stream);

/* zero_fsdp_linear_forward / _backward with the epilogue and its gradient:
     forward:  w_full = all-gather(w_shards); y = act(x W + bias) + residual,
               keeping what the epilogue names.
     backward: w_full again; dz = dy act'(preact); dbias; dx = dz W^T;
               dw_full = x^T dz from the kept x (bf16 or 8 bits), padding
               rows zeroed.  dz is a batch x out bf16 buffer (it may be dy or a
               bf16 preact); for ZERO_ACT_NONE it may be NULL and dy is used as
               it is.  The steps run in this order, and a buffer may be
               written again once nothing later reads it (dx over dy, dw_full
               over w_full); one address for two things that are needed at
               once, or for a result and a shard, is refused.  w_full comes
               before all that the call reads, x and dz are read last, for dW.
               dbias may be NULL; workspace as zero_act_backward.
   batch is any number here; otherwise as zero_fsdp_linear_*. */
zero_status zero_fsdp_linear_act_forward(const zero_layout *layout, int32_t unit,
                                         const uint16_t *const *w_shards, int64_t batch,
                                         const uint16_t *x, uint16_t *w_full,
                                         const zero_epilogue *epilogue, void *y,
                                         int32_t y_dtype, void *stream);
zero_status zero_fsdp_linear_act_backward(const zero_layout *layout, int32_t unit,
                                          const uint16_t *const *w_shards, int64_t batch,
                                          const zero_saved *x, int32_t act,
                                          const zero_saved *preact, const uint16_t *dy,
                                          uint16_t *w_full, uint16_t *dz, void *dx,
                                          int32_t dx_dtype, float *dw_full, float *dbias,
                                          float *workspace, int64_t n_workspace, void *stream);

/* An FSDP expert layer: unit `unit` of a row layout holds n_experts weights
   of in x out one after the other (rows = n_experts * in, cols = out), sharded
   by rows like any other unit.
     forward:  w_full = all-gather; y = the grouped product of x by rows.
     backward: w_full again; dx = grouped dy W_e^T; dw_full = the experts' dW
               one after the other (fp32, the padded unit), ready for
               zero_reduce_shard and zero_adam_step.
   in and out multiples of 8; w_full needs memory apart from all that a call
   reads, dx apart from x, dy and dw_full.  Rows in no group keep their y and
   dx. */
zero_status zero_fsdp_experts_forward(const zero_layout *layout, int32_t unit,
                                      int32_t n_experts, const uint16_t *const *w_shards,
                                      const int64_t *offsets, int64_t rows, const uint16_t *x,
                                      uint16_t *w_full, const zero_epilogue *epilogue, void *y,
                                      int32_t y_dtype, void *stream);
zero_status zero_fsdp_experts_backward(const zero_layout *layout, int32_t unit,
                                       int32_t n_experts, const uint16_t *const *w_shards,
                                       const int64_t *offsets, int64_t rows, const uint16_t *x,
                                       const uint16_t *dy, uint16_t *w_full, void *dx,
                                       int32_t dx_dtype, float *dw_full, void *stream);

/* --------------------------------------------- training operators -- */

/* What a rank's training pass does between its linear layers and around them:
   layer norm, routing to experts and moving their rows, the loss of a linear head,
   and the optimizer step of parameters that are tensors of their own, as FSDP2
   keeps them.  Everything under CONVENTIONS holds here; a matrix without rows or
   columns is never read, and its address may be NULL.  One address for two
   things that a call needs at once is refused, the in-place forms named below
   excepted. */

/* Layer norm of rows of `cols` values: with mu and var a row's mean and variance
   (about the mean, over cols) and r = 1 / sqrt(var + eps),
       y = (x - mu) r gain + bias.
   x and y bf16 or fp32; gain and bias cols values of param_dtype, each may be NULL
   (1, 0); mean and rstd receive mu and r (fp32, rows each; may be NULL).  y may be
   x (same type and leading dimension).  eps >= 0.  Fewer than 2^31 rows, or 2^22 of
   more than 16384 columns, here and in the gradient. */
zero_status zero_layer_norm_forward(int64_t rows, int64_t cols, const void *x, int64_t ldx,
                                    int32_t x_dtype, const void *gain, const void *bias,
                                    int32_t param_dtype, float eps, void *y, int64_t ldy,
                                    int32_t y_dtype, float *mean, float *rstd, void *stream);

/* Its gradient, from the kept x, mean and rstd: with xh = (x - mu) r, h = dy gain,
       dx    = r (h - mean(h) - xh mean(h xh)) + residual   (means over the row)
       dgain = sum over rows of dy xh,  dbias = sum over rows of dy   (fp32).
   residual (rows x cols of dx's type, leading dimension ldr; NULL: 0) is the
   gradient that reaches x past the norm.  dx may be dy, x or the residual (same type
   and leading dimension).  dgain and dbias may be NULL; either needs `workspace` of
   zero_layer_norm_workspace(rows, cols) floats (at most 512 cols), used until the
   call's work has run: calls that overlap in time, and captured graphs that do, need
   one each.  The sums run in a fixed order; over several rows they take fewer than
   2^27 columns.  rows = 0 writes zeros to both. */
zero_status zero_layer_norm_backward(int64_t rows, int64_t cols, const void *dy, int64_t lddy,
                                     int32_t dy_dtype, const void *x, int64_t ldx,
                                     int32_t x_dtype, const void *gain, int32_t param_dtype,
                                     const float *mean, const float *rstd, const void *residual,
                                     int64_t ldr, void *dx, int64_t lddx, int32_t dx_dtype,
                                     float *dgain, float *dbias, float *workspace,
                                     int64_t n_workspace, void *stream);
int64_t zero_layer_norm_workspace(int64_t rows, int64_t cols);

/* How tokens choose experts.  s = softmax or sigmoid of a token's n_experts logits.
   Experts are ranked by s + bias, or by the logit where there is no bias (which
   ranks as s does), the lower number first among equals, NaN last.  With n_groups
   > 1 the experts fall into that many runs of equal length; a group is ranked by its
   best expert (group_best 1) or by the sum of its two best (2; of s where there is
   no bias), and only the top_groups best groups' experts are left.  The token
   takes the top_k best, with weights
       w_j = scale s_j,   or   scale s_j / (sum of the chosen s + 1e-20)
   with `renormalize`.  The bias ranks and does not weigh.  A row of -inf alone has
   scores of 0.  Sums that rank are compared in fp64, to 42 bits.  At most 1024
   experts, 16 of them for a token, 64 groups. */
typedef enum zero_score { ZERO_SCORE_SOFTMAX = 0, ZERO_SCORE_SIGMOID = 1 } zero_score;

typedef struct zero_router {
    int32_t n_experts;
    int32_t top_k;
    int32_t n_groups;   /* 1: no groups; divides n_experts */
    int32_t top_groups; /* 1 .. n_groups; their experts are at least top_k */
    int32_t group_best; /* 1 or 2 */
    int32_t score;      /* zero_score */
    int32_t renormalize;
    float scale;
} zero_router;

/* Routes `tokens` rows of logits (tokens x n_experts, bf16 or fp32).  bias: n_experts
   fp32 or NULL; active: one byte a token or NULL; a token whose byte is 0 takes no
   expert.  Results:
     experts  tokens x top_k int32, the best first; -1 for a token that is not active;
     weights  tokens x top_k fp32; 0 there;
     offsets  n_experts + 1 int64: expert e's rows are offsets[e] .. offsets[e + 1] - 1,
              as the grouped products take them;
     rows_of  tokens x top_k int32: each choice's row when the rows are sorted by expert
              and, within an expert, by token; -1 there.
   workspace: zero_route_workspace int32 (0 for one block's tokens, when it may be
   NULL), used until the call's work has run.  tokens x top_k is below 2^31, and tokens
   at most 2^29 - 64, with groups 2^28 - 16.
   tokens = 0 writes zero offsets. */
zero_status zero_route_forward(const zero_router *router, int64_t tokens, const void *logits,
                               int64_t ldl, int32_t logits_dtype, const float *bias,
                               const uint8_t *active, int32_t *experts, float *weights,
                               int64_t *offsets, int32_t *rows_of, int32_t *workspace,
                               int64_t n_workspace, void *stream);
int64_t zero_route_workspace(const zero_router *router, int64_t tokens);

/* The gradient of the weights with respect to the logits, the choice held fixed:
   dlogits (tokens x n_experts, bf16 or fp32; it may be logits) from dweights
   (tokens x top_k).  `experts` as zero_route_forward left them; numbers outside
   [0, n_experts) count as none, and a token without experts has a gradient of 0.  No
   expert is named twice for a token. */
zero_status zero_route_backward(const zero_router *router, int64_t tokens, const void *logits,
                                int64_t ldl, int32_t logits_dtype, const int32_t *experts,
                                const float *dweights, void *dlogits, int64_t ldd,
                                int32_t dlogits_dtype, void *stream);

/* Tokens' rows to their experts and back.  rows_of is tokens x top_k (top_k at most
   16, tokens x top_k below 2^31); numbers outside [0, rows) are none, and no row is named
   twice (what dispatch and combine_backward leave in such a row is unspecified).
     dispatch          out[rows_of[t][j]] = w[t][j] x[t]   (bf16; weights NULL: copies).
                       Rows that no token has are left as they were.
     combine           y[t] = sum over j of w[t][j] in[rows_of[t][j]] + residual[t], in
                       fp32, rounded once (y bf16 or fp32; weights NULL: 1; residual
                       bf16 or NULL, it may be y).  With weights NULL it is the gradient
                       of dispatch.
     combine_backward  din[rows_of[t][j]] = w[t][j] dy[t] (it may be in) and
                       dweights[t][j] = sum over the columns of dy[t] in[rows_of[t][j]]
                       (fp32; 0 for none), in one pass. */
zero_status zero_experts_dispatch(int64_t tokens, int32_t top_k, int64_t cols, const uint16_t *x,
                                  int64_t ldx, const int32_t *rows_of, const float *weights,
                                  int64_t rows, uint16_t *out, int64_t ldo, void *stream);
zero_status zero_experts_combine(int64_t tokens, int32_t top_k, int64_t cols, const uint16_t *in,
                                 int64_t ldi, int64_t rows, const int32_t *rows_of,
                                 const float *weights, const uint16_t *residual, int64_t ldr,
                                 void *y, int64_t ldy, int32_t y_dtype, void *stream);
zero_status zero_experts_combine_backward(int64_t tokens, int32_t top_k, int64_t cols,
                                          const uint16_t *dy, int64_t lddy, int64_t rows,
                                          const int32_t *rows_of, const float *weights,
                                          const uint16_t *in, int64_t ldi, uint16_t *din,
                                          int64_t lddi, float *dweights, void *stream);

/* Softmax cross entropy of a linear head: z = x W over `vocab` words, x rows x hidden
   bf16, W hidden x vocab (w_order ZERO_K_OUTER, as a linear layer keeps it) or vocab x
   hidden (ZERO_K_INNER, as an embedding does) bf16.  The logits never reach memory.
     lse[r]  = log(sum over c of exp z[r][c]),  loss[r] = lse[r] - z[r][targets[r]];
     dz      = (exp(z - lse) - [c = target]) dloss[r], rounded to bf16 once divided by the
               mantissa of a counted row's dloss, which dx and dw are multiplied by
               (a piece of the vocabulary at a time, in the workspace): in fp32 dx and
               dw are then 1e-4 off or less, in the 2-norm, where all counted rows have
               one dloss, 2e-3 where each has its own;
     dx      = dz W^T (rows x hidden), dw = x^T dz (as W lies), fp32 sums, bf16 or fp32.
   A target outside [0, vocab) is none: loss 0, dx 0, and a dz of 0 in dw, which makes
   a row of x that is not finite NaN there all the same.  hidden and the leading
   dimensions of x and W are multiples of 8, a vocabulary stored as columns too; x and
   W 16-byte aligned; limits of zero_gemm_bf16, and at most 2^26 - 16 rows.  loss, lse
   and dloss are fp32, one a row; lse is what the loss left.  piece: words at a time, 0
   or a multiple of 256; 0 takes the widest pieces of at most ZERO_XENT_PIECE_ELEMS dz
   (and at least 4096 words).  workspace: zero_linear_xent_workspace floats of the pass
   (`backward`; 16-byte aligned), used until the call's work has run.  rows = 0 writes
   zeros to dw. */
#define ZERO_XENT_PIECE_ELEMS 67108864
zero_status zero_linear_xent_forward(int64_t rows, int64_t vocab, int64_t hidden,
                                     const uint16_t *x, int64_t ldx, const uint16_t *w,
                                     int64_t ldw, int32_t w_order, const int64_t *targets,
                                     float *loss, float *lse, float *workspace,
                                     int64_t n_workspace, void *stream);
zero_status zero_linear_xent_backward(int64_t rows, int64_t vocab, int64_t hidden,
                                      const uint16_t *x, int64_t ldx, const uint16_t *w,
                                      int64_t ldw, int32_t w_order, const int64_t *targets,
                                      const float *lse, const float *dloss, void *dx,
                                      int64_t lddx, int32_t dx_dtype, void *dw, int64_t lddw,
                                      int32_t dw_dtype, int64_t piece, float *workspace,
                                      int64_t n_workspace, void *stream);
int64_t zero_linear_xent_workspace(int64_t rows, int64_t vocab, int64_t hidden, int32_t backward,
                                   int64_t piece);

/* The head as an FSDP unit: unit `unit` of a row layout is W (hidden x vocab rows x
   cols for ZERO_K_OUTER, vocab x hidden for ZERO_K_INNER).  Both gather w_full
   first; the backward pass leaves dw_full as the padded unit in fp32 (padding rows
   zeroed), ready for zero_reduce_shard and zero_adam_step.  x, dx: batch x hidden. */
zero_status zero_fsdp_head_forward(const zero_layout *layout, int32_t unit,
                                   const uint16_t *const *w_shards, int32_t w_order,
                                   int64_t batch, const uint16_t *x, uint16_t *w_full,
                                   const int64_t *targets, float *loss, float *lse,
                                   float *workspace, int64_t n_workspace, void *stream);
zero_status zero_fsdp_head_backward(const zero_layout *layout, int32_t unit,
                                    const uint16_t *const *w_shards, int32_t w_order,
                                    int64_t batch, const uint16_t *x, uint16_t *w_full,
                                    const int64_t *targets, const float *lse,
                                    const float *dloss, void *dx, int32_t dx_dtype,
                                    float *dw_full, int64_t piece, float *workspace,
                                    int64_t n_workspace, void *stream);

/* Adam / AdamW over many tensors at once: per element the update of zero_adam_step
   (the same bits, with fp32 states), each tensor with buffers of its own.  A host
   array of descriptions, read during the call:
     n           elements (0: nothing, the pointers may be NULL);
     master      fp32; grad: grad_dtype, multiplied by *clip_coef (device float, NULL:
                 1); param: bf16, receives the new master (NULL: left out);
     m, v        fp32 (ZERO_STATE_FP32), or one code a byte (ZERO_STATE_E4M3) with
                 m_scales, v_scales of ceil(n / 32) bytes;
     decay       0: weight decay is left out for this tensor.
   Different tensors' buffers must not overlap.
   ZERO_STATE_E4M3 keeps m, and the root of v, as e4m3 codes of blocks of 32
   neighbouring elements: a byte b stands for 2^(b - 127), b - 127 the least e in
   [-117, 120] for which the block's largest finite magnitude is at most 448 * 2^e; NaN
   and infinities become NaN.  All-zero buffers are zero states.  A new state is
   rounded to one of the two codes around it at random, by 16 random bits, so that
   averages that move by less than a code's step keep moving; a v above 0 keeps a
   code above 0.  The update itself uses the unrounded m and v, its quotient within
   2^-20 of the one that fp32 states take (their roundings one by one).  The random bits
   depend on `seed`, the step's number and the element's number alone (elements are
   numbered through the list, each tensor from the next multiple of 32): another
   seed for each rank is a good choice.  With bf16 gradients a step moves 16 1/8 bytes
   an element, 28 with fp32 states; master, m and v hold 6 1/16, and 12. */
typedef enum zero_state_format { ZERO_STATE_FP32 = 0, ZERO_STATE_E4M3 = 1 } zero_state_format;

typedef struct zero_tensor {
    int64_t n;
    float *master;
    const void *grad;
    uint16_t *param;
    void *m;
    void *v;
    uint8_t *m_scales;
    uint8_t *v_scales;
    int32_t decay;
} zero_tensor;

zero_status zero_adam_tensors(int32_t n_tensors, const zero_tensor *tensors, int32_t state_format,
                              int32_t grad_dtype, const zero_adam_cfg *cfg, uint64_t seed,
                              const float *clip_coef, void *stream);

/* zero_adam_tensors with the scalars of table[*step_counter - 1] and *step_counter as
   the step's number, both on the device, as zero_adam_step_table takes them: for
   captured steps.  A counter outside [1, n_entries] leaves every buffer untouched. */
zero_status zero_adam_tensors_table(int32_t n_tensors, const zero_tensor *tensors,
                                    int32_t state_format, int32_t grad_dtype,
                                    const zero_adam_table_entry *table, int64_t n_entries,
                                    const int64_t *step_counter, uint64_t seed,
                                    const float *clip_coef, void *stream);

/* The tensors' gradients' sums of squares for zero_clip_coef: fp64 partial sums, one
   for each 8192 elements of a tensor, zero_tensors_partials_count of them. */
zero_status zero_tensors_sumsq(int32_t n_tensors, const zero_tensor *tensors, int32_t grad_dtype,
                               double *partials, int64_t n_partials, void *stream);
int64_t zero_tensors_partials_count(int32_t n_tensors, const zero_tensor *tensors);

/* What n 8-bit state codes and their scales stand for: m, or with `second` v (the
   square of what is kept), bf16 or fp32, both exact but for a v below 2^-126, the
   least normal number, or past the largest. */
zero_status zero_adam_state_read(int64_t n, const uint8_t *codes, const uint8_t *scales,
                                 int32_t second, void *out, int32_t out_dtype, void *stream);

/* ---------------------------------------------------------- errors -- */

const char *zero_status_str(zero_status status);
const char *zero_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* ZERO_SHARD_H */
