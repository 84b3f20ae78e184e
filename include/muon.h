/*
 * muon.h -- C ABI of the MI355X (gfx950) Muon optimizer-step library.
 *
 * One call of muon_step runs one Muon optimizer step over a group of 2-D
 * matrices on one GPU, stream-ordered, with no host synchronisation:
 *
 *   K1  momentum lerp + Nesterov blend + per-block Frobenius reduction +
 *       copy into the wide orientation (bf16 or fp32)         (HBM-bound)
 *   K2  Newton-Schulz, 'standard' or 'gram' form, as grouped MFMA GEMMs
 *       with the quintic fused into their epilogues            (MFMA-bound)
 *   K3  transpose back, shape scale, owned-slice scatter into the fp32 flat
 *       partitions, padding untouched                           (HBM-bound)
 *
 * What the step computes comes from the DeepSpeed pull-request pages it is
 * built from, cited by title and section:
 *   [8526] "Support Muon in BF16_Optimizer with FP32 gradient accumulation",
 *          description (fp32 momentum; Muon on the original matrices; only
 *          each rank's owned intersection is copied into its fp32 partition;
 *          alignment padding excluded; unsupported set-ups rejected up front).
 *   [8600] "Run Muon once per optimizer step under ZeRO-3, not once per
 *          micro-batch", "The problem" / "The change" (once per step on the
 *          accumulated gradient, after the overflow check and before the
 *          norm; Newton-Schulz once per matrix per step; full-shape gradients
 *          passed with each parameter's flat offset) and review thread (the
 *          per-matrix routine takes momentum, beta, the method 'standard' or
 *          'gram' and a per-parameter head count).
 *   [8464] "Fix Muon optimizer under ZeRO CPU offload and bound gather
 *          buffers", momentum-dtype commit (momentum in the fp32 master
 *          dtype; padded final partitions).
 * The numeric form (lerp momentum, Nesterov blend, Frobenius normalisation,
 * quintic coefficients, wide orientation, shape scale sqrt(max(1,rows/cols)))
 * is the plain reading of that prose; the library's design notes list every
 * reading.
 *
 * Conventions for every entry point:
 *  - Every function returns a muon_status; nothing crosses the ABI as an
 *    exception or abort.  All argument checks run before anything is
 *    enqueued, so a call that fails has no side effects.  Asynchronous device
 *    errors surface as MUON_ERR_HIP at a later call or at the caller's own
 *    synchronisation.  muon_last_error() gives a thread-local detail text.
 *  - Pointer tables (grads, momenta, partitions, updates, acc, grad_mb) are
 *    HOST arrays whose elements are DEVICE pointers owned by the caller.
 *    The library never allocates device memory: the caller supplies every
 *    buffer and the workspace.
 *  - Matrices are dense row-major rows x cols in their original orientation.
 *    Only element alignment is required.
 *  - `stream` is a hipStream_t (NULL = the null stream).  Work is ordered on
 *    it; no call synchronises the host.  A plan is not thread-safe; distinct
 *    plans are independent.
 *  - NaN or Inf inputs are not checked; they propagate to the outputs.
 */
#ifndef MUON_MI355X_H
#define MUON_MI355X_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MUON_OK = 0,
  MUON_ERR_INVALID_ARG = 1, /* null pointer, bad size or unknown enum value   */
  MUON_ERR_UNSUPPORTED = 2, /* a configuration this library does not handle   */
  MUON_ERR_LAYOUT = 3,      /* flat ranges overlap or exceed the partitions   */
  MUON_ERR_ALIAS = 4,       /* buffers given to one call overlap              */
  MUON_ERR_WORKSPACE = 5,   /* workspace missing, too small or misaligned     */
  MUON_ERR_HIP = 6          /* a HIP runtime call failed                      */
} muon_status;

typedef enum { MUON_NS_STANDARD = 0, MUON_NS_GRAM = 1 } muon_ns_method;

/* Arithmetic of Newton-Schulz.  FP32: fp32 operands and accumulation
 * throughout.  BF16: bf16 MFMA operands with fp32 accumulation; the Gram
 * form's small-side chain (R, P, Q) is fp32 for blocks with m < 256 and a
 * split-bf16 pair (hi + lo, three bf16 products per product) for m >= 256,
 * except that blocks with m >= 2048 accumulate Q with one bf16 product.
 * Blocks with 64 <= m <= 128 (either form) run their whole iteration in one
 * workgroup; there the Gram form's output product takes Q as a bf16 pair
 * (hi + lo) rather than its bf16 value. */
typedef enum { MUON_PREC_FP32 = 0, MUON_PREC_BF16 = 1 } muon_ns_precision;

/* How the Newton-Schulz products of blocks with m >= 256 (bf16) are put on
 * the device.  LAUNCHES: one launch per product of the schedule over every
 * such block of a wave.  PERSISTENT: one launch per wave runs every product
 * of every such block: a workgroup per CU takes tiles from a queue of its
 * XCD, each block's products stay on one XCD, and a tile starts once its
 * block's previous product is complete (a counter per block), so no
 * device-wide barrier separates the products.  Results are bitwise those
 * of LAUNCHES.  PERSISTENT falls back to LAUNCHES on a device that does not
 * have 8 XCDs of 32 CUs.  Neither form is fixed by the pages, which run the
 * products as framework matmuls; LAUNCHES is the faster one on MI355X for
 * the groups measured, and is the default. */
typedef enum { MUON_SCHED_LAUNCHES = 0, MUON_SCHED_PERSISTENT = 1 } muon_ns_schedule;

/* Storage type of a gradient or update buffer. */
typedef enum { MUON_DT_FP32 = 0, MUON_DT_BF16 = 1 } muon_dtype;

/* One matrix of the group.  num_heads 0 or 1 = one Newton-Schulz block;
 * h > 1 = h equal contiguous row blocks, each orthogonalised on its own
 * ([8600] review thread: the head count is the parameter's own).  flat_offset
 * = index of element (0,0) in the group's flat index space, which the
 * partitions cut into num_partitions pieces of partition_numel elements. */
typedef struct {
  int64_t rows;
  int64_t cols;
  int32_t num_heads;
  int32_t reserved; /* must be 0 */
  int64_t flat_offset;
} muon_matrix;

typedef struct {
  float beta;          /* momentum coefficient, in [0, 1)                  */
  int32_t nesterov;    /* 1: u = (1-beta) G + beta m_new;  0: u = m_new    */
  int32_t method;      /* muon_ns_method                                   */
  int32_t ns_steps;    /* >= 0                                             */
  float a, b, c;       /* quintic coefficients, the same at every step     */
  float eps;           /* X <- u / (||u||_F + eps), per block              */
  int32_t precision;   /* muon_ns_precision                                */
  int32_t grad_dtype;  /* muon_dtype of the grads given to muon_step       */
  uint64_t max_inflight_bytes; /* cap on the workspace's data; 0 = no cap  */
  int32_t schedule;    /* muon_ns_schedule                                 */
  int32_t reserved;    /* must be 0                                        */
} muon_options;

typedef struct {
  int64_t partition_numel; /* elements per partition (P), > 0          */
  int32_t num_partitions;  /* R, > 0                                   */
  int32_t reserved;        /* must be 0                                */
} muon_layout;

/* Host-side counters.  The host never reads a device skip flag, so a step
 * enqueued with one is counted in steps and ns_invocations whether or not
 * the flag later discards it on the device; flagged_steps says how many of
 * the counted steps were such conditional ones.  For a run whose flags all
 * held 0 the counts are exact: ns_invocations = matrices x steps ([8600]
 * "The problem" results table: once per matrix per optimizer step). */
typedef struct {
  uint64_t steps;          /* muon_step / muon_step_ex calls that enqueued */
  uint64_t ns_invocations; /* Newton-Schulz runs enqueued: one per matrix  */
                           /* per counted step                             */
  uint64_t accumulations;  /* muon_accumulate calls that enqueued work     */
  uint64_t waves;          /* workspace waves per step (>= 1)              */
  uint64_t flagged_steps;  /* counted steps enqueued with a skip flag      */
} muon_stats;

/* A contiguous owned intersection of one matrix with one partition:
 * elements [first, first+length) of the row-major flattened matrix go to
 * partitions[partition][offset .. offset+length). */
typedef struct {
  int32_t matrix;
  int32_t partition;
  int64_t offset;
  int64_t first;
  int64_t length;
} muon_run;

/* One Newton-Schulz problem of a plan (a whole matrix or one head block),
 * in its wide orientation m <= n. */
typedef struct {
  int32_t matrix;
  int32_t head;
  int32_t m, n;
  int32_t transposed; /* 1 if the block has more rows than columns */
  int32_t wave;
  double flops;       /* nominal Newton-Schulz flops of this problem */
} muon_problem_info;

/* The default workspace cap: groups needing more run in waves (measured on
 * MI355X: no slower for the Llama-7B and per-head groups, faster for the
 * 70B share, against one wave). */
#define MUON_DEFAULT_INFLIGHT_BYTES ((uint64_t)24 << 30)

typedef struct muon_plan muon_plan;

/* Default options: beta 0.95, Nesterov on, standard form, 5 steps,
 * (a,b,c) = (3.4445, -4.7750, 2.0315), eps 1e-7, bf16 precision, bf16
 * grads, the workspace's data capped at MUON_DEFAULT_INFLIGHT_BYTES (24 GiB:
 * a larger group runs in waves), one launch per product.  Errors: INVALID_ARG if out is NULL. */
muon_status muon_default_options(muon_options *out);

/* Build a plan for a group of n matrices (host only; no device call).
 * The layout is static and computed once ([8526] review thread: split
 * tables computed at init).  Rejected: n < 1; rows or cols < 1; rows or cols
 * beyond 2^31-1; num_heads < 0 or not dividing rows; ns_steps < 0; beta
 * outside [0,1); unknown enums; reserved != 0 (INVALID_ARG / UNSUPPORTED);
 * flat ranges that overlap or leave [0, R*P) (LAYOUT).  On success *out owns
 * host memory only, released by muon_plan_destroy. */
muon_status muon_plan_create(muon_plan **out, const muon_matrix *mats, int32_t n,
                             const muon_options *opt, const muon_layout *layout);

/* Device workspace muon_step needs, in bytes (256-byte aligned base).  The
 * caller allocates it: the library holds no device memory of its own, in
 * place of the gather-buffer cache ([8464] "Changes": cached gather buffers
 * capped at 256 MB and freed on destroy).  With opt.max_inflight_bytes set
 * (as by default) it is proportional to the matrices in flight, not to the
 * whole group
 * ([8526] description: temporary memory proportional to the largest Muon
 * group).  Errors: INVALID_ARG for NULL. */
muon_status muon_plan_workspace_bytes(const muon_plan *p, size_t *bytes);

/* Gradient accumulation into fp32 ([8526] description; [8600] "The change":
 * the partitions accumulate the raw gradient, Muon runs only at the step).
 * acc[i] (fp32, rows x cols) = grad_mb[i] if first != 0, else
 * acc[i] + grad_mb[i].  mb_dtype: muon_dtype of grad_mb.  Runs no
 * Newton-Schulz and touches no momentum.  ws/ws_bytes: the plan's workspace
 * (it holds the launch table).  Errors: INVALID_ARG (null tables or
 * entries, unknown dtype), ALIAS (any two buffers of the call overlap),
 * WORKSPACE, HIP. */
muon_status muon_accumulate(muon_plan *p, float *const *acc, const void *const *grad_mb,
                            int32_t mb_dtype, int32_t first, void *ws, size_t ws_bytes,
                            void *stream);

/* One Muon step over the whole group ([8600] "The change": once per
 * optimizer step, on the accumulated gradient; call it only for steps the
 * overflow check keeps, so a discarded step leaves momentum untouched).
 *   grads[i]      read only, rows x cols, opt.grad_dtype
 *   momenta[i]    fp32 rows x cols, updated in place
 *   partitions[r] fp32, partition_numel each; written only on the owned
 *                 intersections of the matrices, never on padding
 *   ws, ws_bytes  device workspace of at least muon_plan_workspace_bytes,
 *                 256-byte aligned; its contents need not be preserved
 *                 between calls
 * Errors: INVALID_ARG (null table or entry), ALIAS (any two buffers of the
 * call overlap, the workspace included), WORKSPACE (too small / unaligned),
 * HIP (a launch failed). */
muon_status muon_step(muon_plan *p, const void *const *grads, float *const *momenta,
                      float *const *partitions, void *ws, size_t ws_bytes, void *stream);

/* muon_step with the two inputs a mixed-precision training loop adds
 * ([8600] "The change": Muon runs after the overflow check, so a step the
 * loss scaler discards leaves the momentum untouched; [8464] commits:
 * results are checked to agree across loss scales):
 *   skip_flag   DEVICE pointer to an int32, or NULL.  The kernels read it
 *               when they run: non-zero = a discarded step, and nothing
 *               outside the workspace is written (momenta and partitions
 *               keep their contents).  The host never waits for it, so the
 *               plan's counters still count the call (see muon_stats).
 *   grad_scale  multiplies every gradient element before the momentum blend,
 *               in fp32 (1/S for gradients produced under loss scale S);
 *               1.0f gives muon_step bit for bit.  Must be finite.
 * It also leaves, in the workspace, the per-chunk sums of squares of the
 * values written to the partitions, for muon_apply_update.
 * Errors: as muon_step; INVALID_ARG for a non-finite grad_scale, ALIAS if
 * skip_flag overlaps another buffer. */
muon_status muon_step_ex(muon_plan *p, const void *const *grads, float *const *momenta,
                         float *const *partitions, const int32_t *skip_flag, float grad_scale,
                         void *ws, size_t ws_bytes, void *stream);

/* For callers that cannot allocate device memory (a serving loop that may
 * not call hipMalloc, a harness that forbids allocation, code that wants no
 * caller workspace at all): muon_step_ex with the same kernels, arguments
 * and results, minus the workspace.  Its workspace is a device array of
 * MUON_NOALLOC_SCRATCH_BYTES compiled into the library; each GPU the library
 * runs on holds one copy from the first call on it until the process ends.
 * The launch tables reach that array as kernel arguments (at most 96 KB of
 * tables, copied by the runtime at launch), so the call allocates nothing:
 * no hipMalloc, hipHostMalloc or hipFree, and no host heap on success.
 *   - Every call on one GPU shares that GPU's array, which keeps the last
 *     call's contents; the step writes every byte it later reads, so nothing
 *     needs clearing between calls.  Calls that can overlap on one GPU (two
 *     streams, two host threads) race on it: the caller orders them.
 *   - The update-norm partials it leaves stay in the array, so
 *     muon_apply_update cannot follow it (it reports that no step ran on its
 *     workspace); run muon_step_ex when the parameter update follows.
 *   - It enqueues kernels only (no copy, memset or event), so it can be
 *     captured into a graph on a capturing stream: the tables travel in the
 *     captured kernel arguments and each replay uploads them again.  The
 *     plan's counters (muon_plan_stats) count the capture, not the replays.
 * Errors: WORKSPACE if the plan's workspace (muon_plan_workspace_bytes)
 * exceeds MUON_NOALLOC_SCRATCH_BYTES (max_inflight_bytes can cut it into
 * waves that fit); UNSUPPORTED if its tables exceed 96 KB; then as
 * muon_step_ex. */
#define MUON_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
muon_status muon_step_noalloc(muon_plan *p, const void *const *grads, float *const *momenta,
                              float *const *partitions, const int32_t *skip_flag, float grad_scale,
                              void *stream);

/* Overflow check on the step's gradients: *flag (DEVICE int32) = 1 if any
 * element of any grads[i] (rows x cols, `dtype`) is Inf or NaN, else 0.
 * The result can be handed to muon_step_ex / muon_apply_update as their
 * skip flag without a host round trip.  ws/ws_bytes: the plan's workspace
 * (it holds the matrix table).  Errors: INVALID_ARG, ALIAS, WORKSPACE, HIP. */
muon_status muon_check_finite(muon_plan *p, const void *const *grads, int32_t dtype,
                              int32_t *flag, void *ws, size_t ws_bytes, void *stream);

/* The step after the path ([8600] "The change": the gradient norm is taken
 * over the Muon update, clipping semantics unchanged):
 *   norm = sqrt(sum of squares of every owned update element), taken from
 *          the sums the last muon_step / muon_step_ex on this plan and this
 *          workspace left there (fp64, fixed order: deterministic);
 *   clip = max_norm > 0 ? min(1, max_norm / (norm + 1e-6)) : 1;
 *   params[r][j] = params[r][j] * (1 - lr * weight_decay)
 *                  - (lr * clip) * partitions[r][j]      (fp32, one fma)
 * on the owned intersections only; padding untouched.
 *   params[r]      fp32 master partitions, the partitions' layout, updated
 *   partitions[r]  the update as muon_step wrote it, read only
 *   skip_flag      DEVICE int32 or NULL: non-zero = nothing is written
 *   norm_clip_out  DEVICE float[2] or NULL: receives {norm, clip}
 * Call it after the step, with the same workspace and skip flag, before
 * the workspace is used by another step.  Errors: INVALID_ARG (NULL
 * entries, non-finite lr / weight_decay / max_norm, no step on this
 * workspace), ALIAS, WORKSPACE, HIP. */
muon_status muon_apply_update(muon_plan *p, float *const *params, const float *const *partitions,
                              float lr, float weight_decay, float max_norm,
                              const int32_t *skip_flag, float *norm_clip_out, void *ws,
                              size_t ws_bytes, void *stream);

/* The writeback alone (the same kernel muon_step ends with; [8526]
 * description: only the intersection of each matrix's update with a rank's
 * partition is copied there, the alignment padding is not): for every
 * matrix i, partitions[r][...] = fp32(updates[i][j]) * fp32(sqrt(max(1,
 * rows/cols))) on the owned intersections, one IEEE round-to-nearest
 * multiply, padding untouched.  updates[i] is the unscaled Newton-Schulz
 * output in the original orientation, dense rows x cols of dtype `dtype`.
 * ws/ws_bytes: the plan's workspace (it holds the run table).
 * Errors: INVALID_ARG, ALIAS, WORKSPACE, HIP. */
muon_status muon_scatter(muon_plan *p, const void *const *updates, int32_t dtype,
                         float *const *partitions, void *ws, size_t ws_bytes, void *stream);

/* Counters of the plan ([8600] results table counts Newton-Schulz calls). */
muon_status muon_plan_stats(const muon_plan *p, muon_stats *out);

/* Host-side introspection of the static layout (no device call).
 * muon_plan_runs: the owned intersections of matrix `matrix`, in element
 * order; writes min(cap, total) runs and sets *count to the total.
 * muon_plan_problems: the Newton-Schulz problems in plan order, likewise. */
muon_status muon_plan_runs(const muon_plan *p, int32_t matrix, muon_run *out, int32_t cap,
                           int32_t *count);
muon_status muon_plan_problems(const muon_plan *p, muon_problem_info *out, int32_t cap,
                               int32_t *count);

/* Phase timing.  While enabled, muon_step records HIP events on its stream
 * around its three phases (K1 with the norm finalisation; all Newton-Schulz
 * launches; K3), per workspace wave.  muon_plan_phase_ms waits for the last
 * timed step's events and writes the phase times in milliseconds, summed over
 * waves: out[0] K1+norm, out[1] Newton-Schulz, out[2] K3; *ns_launches gets
 * the number of Newton-Schulz launches that step made.  Errors:
 * INVALID_ARG (NULL plan/out, or no timed step yet), HIP. */
muon_status muon_plan_set_timing(muon_plan *p, int32_t enable);
muon_status muon_plan_phase_ms(muon_plan *p, float out[3], int32_t *ns_launches);

void muon_plan_destroy(muon_plan *p);
const char *muon_status_string(muon_status s);
const char *muon_last_error(void);

/* ------------------------------------------------------------------------
 * Operators around the step.  A training program turns token ids into the
 * gradients that muon_accumulate adds up, and logits into a loss and its
 * gradient; these entry points are the parts of that which are neither a
 * matrix product nor the model's own: the embedding lookup and its gradient,
 * the token log-probability, the clipped policy loss, the preference loss
 * and the balance loss of a router.  They need no plan.
 *
 *  - Matrices are row-major with a row stride (`ld`, in elements, at least
 *    the row length); elements are fp32 or bf16 (muon_dtype), whole numbers
 *    int32 or int64 (muon_index_type).  Only element alignment is required.
 *    A buffer of zero elements may be NULL.
 *  - Arithmetic is fp32 an element and fp64 a row (in the balance loss, whose
 *    rows are short, fp32 a token and fp64 the sums over the tokens); bf16
 *    results are rounded once, to nearest even.  No float atomics: results
 *    are bitwise the same from run to run.
 *  - They enqueue kernels only (no copy, memset, event or allocation), so
 *    they can be captured into a graph.
 *  - A workspace is scratch for one call: its contents need not be set
 *    before nor kept after it, and it must not be given to calls that can
 *    overlap in time.
 *  - Errors of all of them: INVALID_ARG (NULL pointer, negative size, ld
 *    below the row length, unknown enum, non-finite factor), UNSUPPORTED (a
 *    size beyond a stated limit), ALIAS (an output overlaps another buffer
 *    of the call, except where in place is allowed; a matrix counts from its
 *    first to its last element, with what lies between its rows), WORKSPACE
 *    (missing, not 256-byte aligned, too small), HIP.
 * ---------------------------------------------------------------------- */

typedef enum { MUON_IDX_INT32 = 0, MUON_IDX_INT64 = 1 } muon_index_type;

/* Embedding lookup: out[t] = scale * table[ids[t]] for t < tokens.  table is
 * vocab x dim, out tokens x dim, both of type `dtype`.  An id outside
 * [0, vocab) (padding) gives a row of zeros.  Limits: tokens, vocab < 2^31. */
muon_status muon_embed_forward(const void *table, int64_t vocab, int64_t dim, int64_t table_ld, int32_t dtype,
                               const void *ids, int32_t id_type, int64_t tokens, float scale, void *out,
                               int64_t out_ld, void *stream);

/* Its gradient by the table, accumulated in fp32 as muon_accumulate does:
 *   acc[v] = (first != 0 ? 0 : acc[v]) + scale * sum of dout[t], ids[t] = v.
 * acc is vocab x dim fp32; with first != 0 every element of it is written
 * (rows without a token get 0), otherwise only rows that have a token are
 * touched.  dout is tokens x dim of type `dtype`.  Ids outside [0, vocab)
 * add nothing.  Limits: tokens, vocab < 2^31. */
muon_status muon_embed_backward_workspace_bytes(int64_t tokens, int64_t vocab, int64_t dim, size_t *bytes);
muon_status muon_embed_backward(const void *ids, int32_t id_type, int64_t tokens, const void *dout, int32_t dtype,
                                int64_t dout_ld, float scale, float *acc, int64_t vocab, int64_t dim, int64_t acc_ld,
                                int32_t first, void *ws, size_t ws_bytes, void *stream);

/* Logits of type `dtype`, rows x vocab, and one target per row, as the
 * three entry points below take them.  A row whose target is outside
 * [0, vocab) has none: it is not read, its log-probability is 0 and so is
 * its gradient.  -inf logits are probabilities of 0; a row with a target
 * and nothing but -inf has lse = -inf and a NaN log-probability; NaN and
 * +inf propagate within their row and the sums it enters.  A term of a loss
 * whose factor is 0 is 0 also where a target of probability 0 makes the
 * rest of it infinite.
 * Limits: rows < 2^31, vocab < 2^29. */
typedef struct {
  const void *logits;
  const void *targets;
  int64_t rows, vocab, ld;
  int32_t dtype;       /* muon_dtype                                     */
  int32_t target_type; /* muon_index_type                                */
} muon_logits;

/* logp[r] = x[r][target] - lse[r], lse[r] = log sum_j exp x[r][j]; fp32.
 * lse may be NULL; both are 0 in rows without a target. */
muon_status muon_token_logprob(const muon_logits *x, float *logp, float *lse, void *stream);

/* The clipped policy loss with a KL term over the rows' targets, and its
 * gradient by the logits:
 *   ratio = exp(logp - old_logp),  J = min(ratio A, clip(ratio, 1 - clip_low, 1 + clip_high) A)
 *   kl = exp(d) - 1 - d,  d = ref_logp - logp
 *   loss = sum_r weights[r] (-J + kl_coef kl)
 * A row of weight 0 counts as one without a target.  old_logp NULL: the
 * rows' own log-probabilities (ratio 1, its gradient kept).  ref_logp NULL:
 * no KL term.  Where both branches of the minimum are equal the gradient is
 * the unclipped one's.  advantages, weights, old_logp, ref_logp: fp32, one
 * a row.
 *   stats[0..4)  loss, its part -sum w J, sum w kl, and the sum of w over
 *                the rows whose clipped branch was the smaller
 *   logp         fp32, one a row (0 in rows that do not count)
 *   dlogits      rows x vocab of x->dtype; may be the logits themselves
 *                (same pointer and ld). */
typedef struct {
  double clip_low, clip_high; /* >= 0 */
  double kl_coef;
} muon_policy_options;
muon_status muon_policy_loss_workspace_bytes(int64_t rows, size_t *bytes);
muon_status muon_policy_loss(const muon_logits *x, const float *advantages, const float *weights,
                             const float *old_logp, const float *ref_logp, const muon_policy_options *opt,
                             float *stats, float *logp, void *dlogits, int64_t dlogits_ld, void *ws, size_t ws_bytes,
                             void *stream);

/* The preference loss of `pairs` pairs of sequences packed into the rows,
 * and its gradient by the logits.  Sequence s has the rows
 * [offsets[s], offsets[s + 1]) (offsets non-decreasing, 2 pairs + 1 of
 * them; what falls outside [0, rows) is cut off); sequences i and pairs + i
 * are the chosen and the rejected one of pair i.
 *   gain_s = sum of the sequence's logp - ref_logp[s],  m = beta (gain_chosen - gain_rejected)
 *   loss = mean over pairs of -(1 - label_smoothing) log sigmoid(m) - label_smoothing log sigmoid(-m)
 *   rewards[s] = beta gain_s
 * Rows of no sequence get a zero gradient.  ref_logp and rewards: fp32,
 * 2 pairs of them; loss: one fp32.  dlogits may be the logits themselves
 * (same pointer and ld).  pairs >= 1, 0 <= label_smoothing <= 1. */
typedef struct {
  double beta, label_smoothing;
} muon_preference_options;
muon_status muon_preference_loss_workspace_bytes(int64_t rows, int64_t pairs, size_t *bytes);
muon_status muon_preference_loss(const muon_logits *x, const void *offsets, int32_t offset_type, int64_t pairs,
                                 const float *ref_logp, const muon_preference_options *opt, float *loss,
                                 float *rewards, void *dlogits, int64_t dlogits_ld, void *ws, size_t ws_bytes,
                                 void *stream);

/* The balance loss of a router with `experts` experts and k choices a token,
 * the tokens each expert gets, and the gradient by the router's logits.  T
 * counts the tokens with valid[t] != 0 (all of them if valid is NULL; at
 * least 1 is divided by):
 *   counts[e] = choices of e among the valid tokens,  f_e = counts[e] / (T k)
 *   balance = experts * sum_e f_e mean_t p[t][e],  z = mean_t lse[t]^2
 *   loss = coef balance + z_coef z
 * p is the softmax of a token's logits, lse its log-sum-exp; the counts
 * carry no gradient.  choices is tokens x k, dense; a choice outside
 * [0, experts) is counted nowhere.  Tokens that are not valid get a zero
 * gradient and are not read.  -inf logits are probabilities of 0; a valid
 * token with nothing else has no softmax: its gradient, the balance and the
 * loss are NaN, and z is infinite.
 *   counts  int32, one an expert;  stats[0..3)  loss, balance, z
 *   dlogits tokens x experts of type `dtype`; may be the logits themselves
 *           (same pointer and ld).
 * Limits: experts <= MUON_BALANCE_MAX_EXPERTS, tokens * k < 2^31. */
#define MUON_BALANCE_MAX_EXPERTS 1024
typedef struct {
  double coef, z_coef;
} muon_balance_options;
muon_status muon_balance_loss_workspace_bytes(int64_t tokens, int64_t experts, size_t *bytes);
muon_status muon_balance_loss(const void *logits, int64_t tokens, int64_t experts, int64_t ld, int32_t dtype,
                              const void *choices, int32_t choice_type, int64_t k, const uint8_t *valid,
                              const muon_balance_options *opt, int32_t *counts, float *stats, void *dlogits,
                              int64_t dlogits_ld, void *ws, size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Operators of a trained layer: dropout, a router's choice of experts, the
 * order of the tokens by expert, the experts' weighted sum, and the product
 * with a weight matrix, or with one a group of rows, each with its
 * gradient.  Conventions and errors as above; what else lies in a matrix's
 * allocation, and rows that a call's definition leaves out, keep their
 * contents.
 * ---------------------------------------------------------------------- */

/* Dropout: out = residual + (kept ? x / (1 - p) : 0), rounded once; residual
 * may be NULL (none).  Element (r, c) is kept if word c mod 4 of
 *   Philox4x32-10, counter (c / 4, r, site, step), key (seed, low half first)
 * is at least round(p 2^32): the mask depends on where an element stands and
 * on seed, site and step alone, and is never stored.  The gradient by x is
 * the same call on the gradient by out, without a residual.  A dropped
 * element adds nothing, also where x is not finite.  If device_step is not
 * NULL its low 32 bits are read on the device instead of step, so that a
 * captured call draws anew whenever the program raises it.  0 <= p < 1.  out
 * may be x or the residual (same pointer and ld). */
muon_status muon_dropout(const void *x, int64_t rows, int64_t cols, int64_t ld, int32_t dtype, double p, uint64_t seed,
                         uint32_t site, uint32_t step, const int64_t *device_step, const void *residual,
                         int64_t residual_ld, void *out, int64_t out_ld, void *stream);

/* A router's choice of k experts a token.
 *   s = softmax or sigmoid of the token's logits, rank = s + bias
 *   With groups > 1 the experts are cut into equal consecutive groups; a
 *   group's value is the sum of its group_top best ranks, and only experts
 *   of the keep_groups groups of highest value can be chosen.
 *   choices[t]  the k experts of highest rank, highest first
 *   weights[t]  scale s_j / (sum of the chosen s + 1e-20), or scale s_j if
 *               renormalize is 0
 * Of equal ranks or values the lower index goes first.  The choice is that
 * of the exact ranks: ranks that fp32 does not tell apart are computed again
 * in fp64.  Without a bias (NULL), and with group_top 1 or one group, experts
 * are ranked by their logits.  An expert whose logit or bias is -inf is never
 * chosen; where a token has fewer than k experts left, and in tokens that are
 * not valid (valid NULL: all are), the choice is -1 and its weight 0.  A NaN
 * ranks below every number.
 * The gradient by the logits, for the gradient dweights by the weights, is
 * written (first != 0) or added to what dlogits holds; the choice itself
 * carries none, nor does the bias.  Choices outside [0, experts) add nothing;
 * tokens that are not valid get zeros, or keep what they hold.  It takes the
 * scoring, renormalize and scale of the choice, and no notice of the groups.
 * Limits: experts <= MUON_BALANCE_MAX_EXPERTS, k <= MUON_ROUTE_MAX_CHOICES,
 * groups <= MUON_ROUTE_MAX_GROUPS, tokens * k < 2^31, and tokens < 2^26 of
 * more than 256 experts. */
typedef enum { MUON_SCORE_SOFTMAX = 0, MUON_SCORE_SIGMOID = 1 } muon_scoring;
#define MUON_ROUTE_MAX_CHOICES 32
#define MUON_ROUTE_MAX_GROUPS 32
typedef struct {
  int32_t scoring;     /* muon_scoring                                    */
  int32_t renormalize;
  int32_t groups, keep_groups;
  int32_t group_top;   /* 1 or 2                                          */
  int32_t reserved;
  double scale;
} muon_route_options;
muon_status muon_route(const void *logits, int64_t tokens, int64_t experts, int64_t ld, int32_t dtype, const float *bias,
                       const uint8_t *valid, const muon_route_options *opt, void *choices, int32_t choice_type,
                       int64_t k, float *weights, void *stream);
muon_status muon_route_backward(const void *logits, int64_t tokens, int64_t experts, int64_t ld, int32_t dtype,
                                const uint8_t *valid, const muon_route_options *opt, const void *choices,
                                int32_t choice_type, int64_t k, const float *dweights, void *dlogits,
                                int64_t dlogits_ld, int32_t first, void *stream);

/* The order of the tokens by expert.  Every choice in [0, experts) gets a
 * slot: those of expert e have the slots [offsets[e], offsets[e + 1]), in the
 * order of their tokens and of a token's choices.
 *   slot_tokens  tokens * k: the slots' tokens, -1 behind the last slot
 *   offsets      experts + 1
 *   place        tokens x k: the choices' slots, -1 for a choice outside
 * With slot_tokens as ids, muon_embed_forward gathers the experts' rows.
 * Limits: experts <= MUON_BALANCE_MAX_EXPERTS, tokens * k < 2^31. */
muon_status muon_expert_order_workspace_bytes(int64_t tokens, int64_t k, int64_t experts, size_t *bytes);
muon_status muon_expert_order(const void *choices, int32_t choice_type, int64_t tokens, int64_t k, int64_t experts,
                              int32_t *slot_tokens, int32_t *offsets, int32_t *place, void *ws, size_t ws_bytes,
                              void *stream);

/* What the experts return, summed up a token:
 *   out[t] = residual[t] + sum_j weights[t][j] y[place[t][j]]
 * y is rows x dim, out and residual tokens x dim, of type `dtype`; place and
 * weights are tokens x k, dense; a place outside [0, rows) adds nothing.
 * weights NULL: 1 each (the gradient of the gather); residual NULL: none.
 * out may be the residual (same pointer and ld).
 * The gradients, for the gradient dout by out:
 *   dy[place[t][j]] = weights[t][j] dout[t]       rows of no place are kept
 *   dweights[t][j]  = sum dout[t] y[place[t][j]]  0 for a place outside
 * Either may be NULL; y is read for dweights only.  dy may be y (same pointer
 * and ld).  No two places may be equal (muon_expert_order gives none).
 * Limits: tokens * k, rows, dim < 2^31, tokens < 2^26, tokens * dim < 2^34. */
muon_status muon_expert_combine(const void *y, int64_t rows, int64_t dim, int64_t y_ld, int32_t dtype,
                                const int32_t *place, int64_t tokens, int64_t k, const float *weights,
                                const void *residual, int64_t residual_ld, void *out, int64_t out_ld, void *stream);
muon_status muon_expert_combine_backward(const void *dout, int64_t tokens, int64_t dim, int64_t dout_ld, int32_t dtype,
                                         const int32_t *place, int64_t k, const float *weights, const void *y,
                                         int64_t y_ld, int64_t rows, void *dy, int64_t dy_ld, float *dweights,
                                         void *stream);

/* The product with a weight matrix and what usually stands around it:
 *   pre = x w + bias,  out = act(pre) + residual
 * x is rows x in, out, pre and residual rows x out, of the weights' type.
 * bias (out numbers a group, dense), pre and residual may be NULL; out may be
 * the residual (same pointer and ld).  act: max(v, 0), v / (1 + exp(-v)), v
 * Phi(v), or v (1 + tanh(sqrt(2 / pi) (v + 0.044715 v^3))) / 2.
 * Every group of rows may have a matrix of its own (a layer's experts): group
 * g has the rows [offsets[g], offsets[g + 1]) (non-decreasing, on the device;
 * what falls outside [0, rows) is cut off).  Rows of no group are not
 * touched.  offsets may be NULL for one group of all rows.
 * Sums are fp32, of bf16 products or of fp32 ones; what leaves is rounded
 * once.
 * Limits, of the gradients too: rows, in, out < 2^31, groups <=
 * MUON_LINEAR_MAX_GROUPS, and with R = rows / 128 + groups, I = in / 128 + 1,
 * O = out / 128 + 1 (rounded down) each of R I, R O and I O groups < 2^23. */
typedef enum {
  MUON_ACT_NONE = 0, MUON_ACT_RELU = 1, MUON_ACT_SILU = 2, MUON_ACT_GELU = 3, MUON_ACT_GELU_TANH = 4
} muon_activation;
typedef enum { MUON_W_IN_OUT = 0, MUON_W_OUT_IN = 1 } muon_w_layout;
#define MUON_LINEAR_MAX_GROUPS 1024
typedef struct {
  const void *w;
  int64_t in, out;
  int64_t ld;           /* of a row: of an input's weights (MUON_W_IN_OUT) or an output's */
  int64_t stride;       /* from a group's matrix to the next one's, in elements           */
  int32_t layout;       /* muon_w_layout                                                  */
  int32_t groups;
  const void *offsets;  /* DEVICE, groups + 1 whole numbers, or NULL                      */
  int32_t offset_type;  /* muon_index_type                                                */
  int32_t dtype;        /* muon_dtype                                                     */
} muon_weights;
muon_status muon_linear_workspace_bytes(int64_t rows, int64_t in, int64_t out, int64_t groups, size_t *bytes);
muon_status muon_linear_forward(const void *x, int64_t rows, int64_t x_ld, const muon_weights *w, const void *bias,
                                int32_t activation, void *pre, int64_t pre_ld, const void *residual,
                                int64_t residual_ld, void *out, int64_t out_ld, void *ws, size_t ws_bytes,
                                void *stream);

/* Its gradient by x, for the gradient dy by the pre of the product:
 *   dx = (dy w') act'(pre) + residual
 * where pre is what the activation before the product took (x = act(pre):
 * the chain reaches the product before without a pass of its own), and the
 * residual a gradient that joins, such as the skip connection's.  dy is rows
 * x out, dx, pre and residual rows x in.  pre is not read without an
 * activation; residual may be NULL, or dx itself (same pointer and ld).
 * Workspace: muon_linear_workspace_bytes(rows, out, in, groups). */
muon_status muon_linear_input_grad(const void *dy, int64_t rows, int64_t dy_ld, const muon_weights *w,
                                   int32_t activation, const void *pre, int64_t pre_ld, const void *residual,
                                   int64_t residual_ld, void *dx, int64_t dx_ld, void *ws, size_t ws_bytes,
                                   void *stream);

/* Its gradients by the weights and the bias, accumulated in fp32 as
 * muon_accumulate does:
 *   dw[g] = (first != 0 ? 0 : dw[g]) + the group's x' dy,  dbias[g] likewise
 * the sums of dy's columns.  dw is laid out by dw_ld, dw_stride and dw_layout
 * as muon_weights; dbias is dense, and may be NULL.  Every element is
 * written, also of groups without rows. */
muon_status muon_linear_weight_grad_workspace_bytes(int64_t rows, int64_t in, int64_t out, int64_t groups, size_t *bytes);
muon_status muon_linear_weight_grad(const void *x, int64_t rows, int64_t in, int64_t x_ld, const void *dy, int64_t out,
                                    int64_t dy_ld, int32_t dtype, const void *offsets, int32_t offset_type,
                                    int64_t groups, float *dw, int64_t dw_ld, int64_t dw_stride, int32_t dw_layout,
                                    float *dbias, int32_t first, void *ws, size_t ws_bytes, void *stream);

/* dpre = dy act'(pre), where a product's activation is not followed by
 * another product.  dpre may be dy or pre (same pointer and ld). */
muon_status muon_activation_grad(const void *dy, int64_t rows, int64_t cols, int64_t dy_ld, int32_t dtype,
                                 int32_t activation, const void *pre, int64_t pre_ld, void *dpre, int64_t dpre_ld,
                                 void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MUON_MI355X_H */
