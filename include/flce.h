/*
 * flce.h -- C ABI of the GB300 (sm_103a) fused linear cross entropy library.
 *
 * The loss of a language-model head and what a training step runs around it:
 *
 *  flce_fwd_bwd  Fused linear cross entropy (FLCE): the lm_head projection
 *                z = H W^T (+ b) fused with softmax cross entropy (ignore_index,
 *                reduction none / sum / mean) and its backward (grad_hidden,
 *                grad_weight, grad_bias), chunked over tokens so the [N, V]
 *                logits never exist.  Defined by "Peak Performance, Minimized
 *                Memory: Optimizing torchtune's performance with torch.compile
 *                & Liger Kernel", section "Introduction to Liger Kernel",
 *                Figure 1 "Fused Linear Cross Entropy" and its four steps
 *                (flatten, project chunk by chunk, partial loss + chunk
 *                logits gradient, hidden gradient + accumulated head
 *                gradient); call shape from the liger-kernel 0.0.1 -> 0.1.1
 *                PyPI diff, README "Compose Your Own Model" (weight, input,
 *                target, then backward).
 *
 *  ce_fwd_bwd    Cross entropy on materialised logits [N, V]: loss and the
 *                logits gradient in one call, the gradient optionally
 *                written over the logits.  Defined by the same README,
 *                "Kernels" list, CrossEntropy item (PyTorch CrossEntropyLoss
 *                semantics, loss and gradient computed together, in-place
 *                replacement of the input); logits dtypes and the reduction /
 *                ignore contract from DeepSpeed PR #8540 (optional Liger
 *                vocab-parallel CE backend), "Changes" and "Real-device
 *                validation".
 *
 *  ln_fwd, ln_bwd  Layer norm, or its form without the mean, in front of the
 *                head: it gives flce_fwd_bwd its hidden states and takes their
 *                gradient.
 *
 *  grad_norm, adamw_step  The norm of all gradients and one AdamW step over
 *                many tensors, with moments in fp32 or in 8 bits.
 *
 *  policy_fwd_bwd, preference_fwd_bwd, distill_fwd_bwd  The losses of
 *                post-training on materialised logits, each with its gradient:
 *                the clipped policy loss with a KL term, the loss over pairs of
 *                sequences, and the distance from a teacher's top logits.
 *
 *  embedding_fwd, embedding_bwd  Rows of a table by token, and the table's
 *                gradient, which may be added to the head's where both share
 *                one weight.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Every tensor pointer is a DEVICE pointer to memory the caller owns.  The
 *    library never allocates, frees or synchronises; all work is enqueued on
 *    `stream` (a cudaStream_t; NULL is the legacy default stream) and runs
 *    asynchronously.  Outputs are valid once the stream reaches the call.
 *  - Matrices are row-major and, where no ld is given, contiguous.  bf16 is
 *    IEEE bfloat16; results stored as bf16 are rounded to nearest even.
 *  - Host-checkable faults (NULL required pointer, bad enum, bad shape or
 *    alignment, workspace too small) return an error code BEFORE anything is
 *    enqueued.  FLCE_ERR_CUDA means a launch failed (cudaGetLastError).
 *  - Device-detected faults never trap.  They are OR-ed as bits into the
 *    device status word: a target outside [0, V) that is not ignore_index sets
 *    FLCE_STATUS_BIT_TARGET_RANGE and that row is treated as ignored; a
 *    pipeline wait that exceeded its time limit sets FLCE_STATUS_BIT_TIMEOUT
 *    and that call's outputs are undefined.  The status word is `status_dev`
 *    when given (never cleared by the library), else the first 4 bytes of the
 *    workspace (cleared at the start of each call).
 *  - Calls that share a workspace must not overlap in time (same stream, or
 *    ordered by events).
 */
#ifndef FLCE_H_
#define FLCE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t, declared here so the header needs no CUDA. */
typedef struct CUstream_st* flce_stream_t;

typedef enum {
  FLCE_REDUCTION_NONE = 0, /* per-row losses [N]                      */
  FLCE_REDUCTION_SUM = 1,  /* sum over valid rows, scalar             */
  FLCE_REDUCTION_MEAN = 2  /* sum / number of valid rows (NaN if 0)   */
} flce_reduction_t;

/* FLCE_DTYPE_FP32_ROUNDED: fp32 FLCE operands rounded to bf16 once (the
 * fast mode of flce_fwd_bwd_typed); not a logits type. */
typedef enum {
  FLCE_DTYPE_BF16 = 0,
  FLCE_DTYPE_FP32 = 1,
  FLCE_DTYPE_FP16 = 2,
  FLCE_DTYPE_FP32_ROUNDED = 3
} flce_dtype_t;

typedef enum {
  FLCE_OK = 0,
  FLCE_ERR_INVALID_ARG = 1,  /* NULL pointer, negative size, bad enum       */
  FLCE_ERR_UNSUPPORTED = 2,  /* dtype or layout not handled (e.g. H % 8)    */
  FLCE_ERR_WORKSPACE = 3,    /* workspace NULL/too small/misaligned         */
  FLCE_ERR_CUDA = 4,         /* a CUDA call or kernel launch failed         */
  FLCE_ERR_TARGET_RANGE = 5, /* value of a device status bit (see above)    */
  FLCE_ERR_TIMEOUT = 6,      /* value of a device status bit (see above)    */
  FLCE_ERR_MISALIGNED = 7    /* a pointer breaks its alignment requirement  */
} flce_status_t;

/* Bits of the device status word. */
#define FLCE_STATUS_BIT_TARGET_RANGE 0x1
#define FLCE_STATUS_BIT_TIMEOUT 0x2
#define FLCE_STATUS_BIT_SEQUENCE_RANGE 0x4

/* Human-readable name of a status code (static storage, never NULL). */
const char* flce_status_string(flce_status_t status);

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
int flce_version(void);

/* ------------------------------------------------------------------------
 * Fused linear cross entropy
 * ------------------------------------------------------------------------ */

/* Token chunk used when flce_fwd_bwd is given chunk = 0, for these sizes. */
int64_t flce_default_chunk(int64_t N, int64_t H, int64_t V);

/* Bytes of workspace flce_fwd_bwd needs for these sizes (chunk 0 = default).
 * It grows with chunk * V (the bf16 logits / grad-logits of one chunk) and
 * with N (4 bytes of per-row loss), never with N * V.  Returns 0 for invalid
 * sizes. */
size_t flce_workspace_size(int64_t N, int64_t H, int64_t V, int64_t chunk, int reduction);

/* flce_workspace_size_typed -- the workspace flce_fwd_bwd_typed needs for
 * operands of `dtype` (flce_dtype_t); 0 for an unknown dtype or invalid
 * sizes. */
size_t flce_workspace_size_typed(int dtype, int64_t N, int64_t H, int64_t V, int64_t chunk,
                                 int reduction);

/*
 * flce_fwd_bwd -- loss and gradients of cross_entropy(hidden @ weight^T + bias, target).
 *
 *  hidden        bf16 [N, H]; 16-byte aligned; H a multiple of 8 (TMA rows).
 *  weight        bf16 [V, H]; 16-byte aligned.
 *  bias          bf16 [V] or NULL (no bias).
 *  target        int64 [N]; class ids in [0, V) or ignore_index.
 *  N, H, V       tokens (>= 0), hidden size (>= 8, % 8 == 0), vocabulary (>= 1).
 *  ignore_index  targets equal to it add no loss and no gradient (checked
 *                before the range check, so it may lie inside [0, V)).
 *  reduction     flce_reduction_t.  Mean divides by the number of valid
 *                targets over all N rows.
 *  chunk         tokens per chunk (>= 1), or 0 for flce_default_chunk.
 *  grad_scale    upstream gradient g of the reduced loss; multiplies every
 *                gradient (1.0 for plain loss.backward()).
 *  grad_out_none fp32 [N] per-row upstream gradients, reduction NONE only
 *                (gradient of sum_n g * grad_out[n] * loss_n); NULL = ones.
 *  loss          fp32 output: [N] for NONE (0 for ignored rows), else [1].
 *  grad_hidden   bf16 [N, H] output (always overwritten), or NULL to skip.
 *  grad_weight   fp32 [V, H] output, 16-byte aligned, or NULL to skip.
 *  grad_bias     fp32 [V] output, or NULL to skip (must be NULL if bias is).
 *  accumulate    0: grad_weight / grad_bias are overwritten; 1: added to.
 *  n_valid_out   int32 [1] output (number of valid targets), or NULL.
 *  lse_out       fp32 [N] output: log-sum-exp of every row's logits, or NULL.
 *  target_logit_out  fp32 [N] output: z[n, target_n] for valid rows, 0 for
 *                ignored rows, or NULL.  (These two are the per-row partials
 *                a vocabulary-parallel caller would combine across shards.)
 *  workspace     device scratch of >= flce_workspace_size(...) bytes,
 *                256-byte aligned; contents on entry are ignored.
 *  status_dev    int32 device status word (see conventions), or NULL.
 *  stream        CUDA stream.
 *
 * Arithmetic: the projection runs on the tensor cores (bf16 x bf16, fp32
 * accumulation); the log-sum-exp and the target logit come from the fp32
 * accumulator; the chunk's grad-logits are rounded to bf16 before the two
 * backward products, which accumulate in fp32.
 */
flce_status_t flce_fwd_bwd(const void* hidden, const void* weight, const void* bias,
                           const int64_t* target, int64_t N, int64_t H, int64_t V,
                           int64_t ignore_index, int reduction, int64_t chunk,
                           float grad_scale, const float* grad_out_none, float* loss,
                           void* grad_hidden, float* grad_weight, float* grad_bias,
                           int accumulate, int32_t* n_valid_out, float* lse_out,
                           float* target_logit_out, void* workspace, size_t workspace_bytes,
                           int32_t* status_dev, flce_stream_t stream);

/*
 * flce_fwd_bwd_typed -- flce_fwd_bwd with the operand type given: dtype is
 *   FLCE_DTYPE_BF16          exactly flce_fwd_bwd;
 *   FLCE_DTYPE_FP16          hidden, weight, bias and grad_hidden are IEEE half;
 *   FLCE_DTYPE_FP32          hidden, weight, bias and grad_hidden are fp32,
 *                            multiplied at about fp32 accuracy (below);
 *   FLCE_DTYPE_FP32_ROUNDED  the same buffers, the operands rounded to bf16
 *                            once (the fast mode, below);
 * everything else is as in flce_fwd_bwd.  The workspace must hold
 * flce_workspace_size_typed(dtype, ...) bytes (the same as
 * flce_workspace_size for the two 16-bit types; FP32 adds bf16 hi + lo
 * copies of hidden and weight and a second plane of chunk logits,
 * FP32_ROUNDED one bf16 copy of hidden, weight and bias).  Other dtypes return
 * FLCE_ERR_UNSUPPORTED.  The logits dtypes FP32 / FP16 / BF16
 * the DeepSpeed PR #8540 description ("optional Liger vocab-parallel CE
 * backend", section "Changes") validates carry over to the fused form here.
 *
 * Arithmetic with fp16: fp16 x fp16 on the tensor cores with fp32
 * accumulation; the chunk logits are kept in fp16, and the chunk's
 * grad-logits are stored in fp16 divided by the part of the gradient scale
 * common to all rows (g / n_valid for MEAN, g for SUM, g * max|grad_out| for
 * NONE), so they lie in [-1, 1] rather than underflowing fp16's range; the
 * two backward products multiply that factor back in fp32.  grad_bias is
 * summed from the fp32 grad-logits.
 *
 * Arithmetic with FP32: hidden and weight are split once per call into bf16
 * hi = round(x) and lo = round(x - hi) (nearest, ties to even), and every
 * product is formed on the tensor cores as hi.hi + hi.lo + lo.hi with fp32
 * accumulation (the dropped lo.lo term is below 2^-16 of each product), at
 * a third of the bf16 tensor rate; the bias is added in fp32; the chunk
 * logits are kept exactly (both halves of their fp32 bits), their gradient
 * is formed in fp32 and split the same way for the two backward products;
 * grad_hidden is written from the fp32 accumulator.
 *
 * Arithmetic with FP32_ROUNDED: hidden, weight and bias are rounded to bf16
 * (to nearest, ties to even) into the workspace once per call and the bf16
 * path runs on those copies, so the loss and grad_weight / grad_bias equal
 * the bf16 entry point's on the rounded inputs; grad_hidden is written from
 * the fp32 accumulator without the bf16 rounding.  This is the rate of the
 * bf16 path at its precision, for callers whose fp32 tensors are master
 * copies of a mixed-precision step.
 */
flce_status_t flce_fwd_bwd_typed(int dtype, const void* hidden, const void* weight, const void* bias,
                                 const int64_t* target, int64_t N, int64_t H, int64_t V,
                                 int64_t ignore_index, int reduction, int64_t chunk,
                                 float grad_scale, const float* grad_out_none, float* loss,
                                 void* grad_hidden, float* grad_weight, float* grad_bias,
                                 int accumulate, int32_t* n_valid_out, float* lse_out,
                                 float* target_logit_out, void* workspace, size_t workspace_bytes,
                                 int32_t* status_dev, flce_stream_t stream);

/* ------------------------------------------------------------------------
 * Cross entropy on materialised logits
 * ------------------------------------------------------------------------ */

/* Bytes of workspace ce_fwd_bwd needs (per-row losses and counters). */
size_t ce_workspace_size(int64_t N, int64_t V, int dtype, int reduction);

/*
 * ce_fwd_bwd -- loss and grad_logits of cross_entropy(logits, target).
 *
 *  logits        [N, V] of `dtype` (FLCE_DTYPE_BF16, FLCE_DTYPE_FP16 or FLCE_DTYPE_FP32).
 *  grad_logits   [N, V] of `dtype` output: scale_n * (softmax - onehot), 0 for
 *                ignored rows.  May equal `logits` (in place: the logits are
 *                consumed) or be a separate buffer (logits left unchanged),
 *                or NULL (loss only).  Partial overlap is not allowed.
 *  target        int64 [N].
 *  ignore_index, reduction, grad_scale, grad_out_none, loss: as flce_fwd_bwd.
 *  workspace     >= ce_workspace_size(...) bytes, 256-byte aligned; contents
 *                on entry are ignored.  One workspace serves one call at a
 *                time (calls on different streams need their own).
 *  status_dev, stream: as flce_fwd_bwd.
 *
 * With 16-byte aligned logits / grad_logits pointers every row length of at
 * least 32 bytes runs on 16-byte vectors (a row that is not a whole number
 * of vectors is handled through its aligned covering range, touching no
 * neighbouring row's elements); otherwise an element-by-element path runs.
 * With N <= 16384 and the vector forms the call is a single kernel launch
 * (no separate counting pass); otherwise a small counting kernel runs
 * first.
 */
flce_status_t ce_fwd_bwd(const void* logits, int dtype, void* grad_logits, const int64_t* target,
                         int64_t N, int64_t V, int64_t ignore_index, int reduction,
                         float grad_scale, const float* grad_out_none, float* loss,
                         void* workspace, size_t workspace_bytes, int32_t* status_dev,
                         flce_stream_t stream);

/* ------------------------------------------------------------------------
 * Vocabulary-parallel building blocks
 * ------------------------------------------------------------------------
 * When the vocabulary is split across shards (tensor parallelism: the
 * vocabulary-parallel cross entropy and the fused lm_head + vocabulary-
 * parallel CE that never builds the [S, B, V/tp] logits -- "Native
 * Liger-Kernel integration in Megatron-LM", PR table and Roadmap item 2;
 * DeepSpeed PR #8540 "Changes"), shard s holds vocabulary ids
 * [vocab_offset, vocab_offset + V_shard).  The cross entropy needs, per row,
 * the log-sum-exp over the whole vocabulary and the target logit; the caller
 * combines the shards' partials (for example with an all-reduce):
 *     lse = M + log(sum_s exp(lse_s - M)),  M = max_s lse_s
 *     z_t = sum_s zt_s              (zt_s is 0 unless shard s holds the target)
 * and then lets every shard form its own gradients from the combined values
 * and per-row scales row_scale[n] = d(reduced loss)/d(loss_n) (0 for ignored
 * rows), which the caller also forms (it knows the global valid count, the
 * reduction and the upstream gradient).  The loss is lse - z_t per row.
 * Targets are global ids; ignore_index marks ignored rows.
 */

/* Bytes of workspace for flce_vp_forward / flce_vp_backward on a chunk of C rows. */
size_t flce_vp_workspace_size(int64_t C, int64_t H, int64_t V_shard);

/* FLCE on one vocabulary shard, forward part, for one chunk of C tokens:
 * projects hidden [C, H] with weight_shard [V_shard, H] (+ bias_shard) into
 * the workspace (bf16) and writes per row lse_shard (fp32 logits), lse16_shard
 * (their bf16 roundings; combine it the same way for the gradient) and
 * target_logit_shard.  The workspace must then be passed, unchanged, to
 * flce_vp_backward for the same chunk.  Alignment and H as flce_fwd_bwd. */
flce_status_t flce_vp_forward(const void* hidden, const void* weight_shard, const void* bias_shard,
                              const int64_t* target, int64_t C, int64_t H, int64_t V_shard,
                              int64_t vocab_offset, int64_t ignore_index, float* lse_shard,
                              float* lse16_shard, float* target_logit_shard, void* workspace,
                              size_t workspace_bytes, int32_t* status_dev, flce_stream_t stream);

/* FLCE on one vocabulary shard, backward part: with lse16 [C] combined over
 * all shards and row_scale [C], forms the shard's logits gradient in the
 * workspace, then grad_hidden_partial (fp32 [C, H], overwritten; the caller
 * sums it over shards), grad_weight_shard (fp32 [V_shard, H]) and
 * grad_bias_shard (fp32 [V_shard]); accumulate = 1 adds to the latter two.
 * Any of the three outputs may be NULL. */
flce_status_t flce_vp_backward(const void* hidden, const void* weight_shard, const int64_t* target,
                               int64_t C, int64_t H, int64_t V_shard, int64_t vocab_offset,
                               int64_t ignore_index, const float* lse16, const float* row_scale,
                               float* grad_hidden_partial, float* grad_weight_shard,
                               float* grad_bias_shard, int accumulate, void* workspace,
                               size_t workspace_bytes, int32_t* status_dev, flce_stream_t stream);

/* Cross entropy on a vocabulary shard of materialised logits [N, V_shard]:
 * per-row partials lse_shard and target_logit_shard.  No workspace. */
flce_status_t ce_vp_partials(const void* logits, int dtype, const int64_t* target, int64_t N,
                             int64_t V_shard, int64_t vocab_offset, int64_t ignore_index,
                             float* lse_shard, float* target_logit_shard, int32_t* status_dev,
                             flce_stream_t stream);

/* ... and the shard's gradient from the combined lse [N] and row_scale [N]:
 * grad = row_scale * (softmax - onehot), written to grad_logits (may equal
 * logits).  No workspace. */
flce_status_t ce_vp_backward(const void* logits, int dtype, void* grad_logits, const int64_t* target,
                             int64_t N, int64_t V_shard, int64_t vocab_offset, int64_t ignore_index,
                             const float* lse, const float* row_scale, int32_t* status_dev,
                             flce_stream_t stream);

/* ------------------------------------------------------------------------
 * Cross entropy on logits without any caller-provided scratch
 * ------------------------------------------------------------------------ */

/* Largest N accepted by ce_fwd_bwd_noalloc. */
#define FLCE_NOALLOC_MAX_ROWS 65536

/*
 * ce_fwd_bwd_noalloc -- the computation of ce_fwd_bwd for callers that cannot
 * allocate device memory or hand over a workspace: for example a plugin whose
 * enqueue step may not allocate, a process whose device memory belongs to
 * another allocator, or a loop that cannot afford cudaMalloc's implicit
 * synchronisation.  The pages have no counterpart; it is an integration aid.
 *
 * Its scratch (256 bytes plus 4 bytes per row) is a fixed device array inside
 * the library, sized for FLCE_NOALLOC_MAX_ROWS rows (about 256 KiB, held by
 * every GPU that loads the library until the process exits).  Arguments are
 * those of ce_fwd_bwd without the workspace; N > FLCE_NOALLOC_MAX_ROWS returns
 * FLCE_ERR_UNSUPPORTED before anything is enqueued.  The entry point calls
 * no allocating routine (no cudaMalloc or cudaFree, no workspace).  Device
 * memory does appear once per device context when the CUDA runtime loads the
 * library's module (the array and the kernels' code; with lazy module
 * loading, the default, this happens at the first call and at the first
 * launch of each kernel): make one warm-up call per device outside any
 * region that must not allocate.
 *
 * The first call on a device context looks the array's device address up (a
 * CUDA runtime query with that device current; again after cudaDeviceReset,
 * whose new context holds the array elsewhere); make that first call before
 * any stream capture.  All calls share the one array: calls that may overlap
 * on the GPU (unordered streams) race and must be serialised by the caller.
 * With status_dev NULL no status is reported.  Like ce_fwd_bwd, a call with
 * N <= 16384 and the vector forms is a single kernel launch.
 */
flce_status_t ce_fwd_bwd_noalloc(const void* logits, int dtype, void* grad_logits,
                                 const int64_t* target, int64_t N, int64_t V,
                                 int64_t ignore_index, int reduction, float grad_scale,
                                 const float* grad_out_none, float* loss, int32_t* status_dev,
                                 flce_stream_t stream);

/* ------------------------------------------------------------------------
 * Layer norm in front of the head
 * ------------------------------------------------------------------------
 * Per row n of x [N, H]:
 *     s    = x (+ residual, rounded to the type of x)
 *     mu   = sum_h s / H            (FLCE_NORM_LAYER; 0 for FLCE_NORM_RMS)
 *     rstd = 1 / sqrt(sum_h (s - mu)^2 / H + eps)
 *     xhat = (s - mu) * rstd,   y = xhat * weight + bias
 * and backward, with u = grad_y * weight:
 *     grad_s = rstd * (u - mean_h(u) [layer only] - xhat * mean_h(u * xhat))
 *     grad_x = grad_residual = grad_s + grad_sum
 *     grad_weight = sum_n grad_y * xhat,   grad_bias = sum_n grad_y
 * Everything between loading and storing is fp32; the rows' sums of squares
 * are taken about the mean, in a second pass over the row held on the chip.
 *
 * Matrices here are rows of H contiguous elements, `ld` elements apart: for an
 * input any ld >= 0 (0 repeats one row), for an output ld >= H, at most 2^29.
 * Pointers need the alignment of their elements only; 16-byte aligned rows
 * (pointer and ld) are the fast case.  Except where said, buffers do not
 * overlap.  An infinity or NaN spoils its own row (and the column sums), no
 * other, and so does an element above 1.8e19 in size, whose square is infinite.
 */
typedef enum {
  FLCE_NORM_LAYER = 0, /* mean and variance                     */
  FLCE_NORM_RMS = 1    /* no mean: the root of the mean square  */
} flce_norm_t;

/*
 * ln_fwd
 *
 *  kind          flce_norm_t.
 *  dtype         type of x, residual, y and sum: FLCE_DTYPE_BF16, _FP16 or _FP32.
 *  residual      [N, H] or NULL: added to x first.
 *  weight, bias  [H] of `param_dtype` (any of the three types), either NULL
 *                (1 and 0).
 *  N, H          rows (>= 0) and columns (1 to 2^24 - 1).
 *  eps           >= 0.
 *  y             [N, H] output.
 *  sum           [N, H] output: s, what the row statistics are taken of, or
 *                NULL (must be NULL without residual).
 *  mean, rstd    fp32 [N] outputs or NULL (mean must be NULL for FLCE_NORM_RMS).
 *
 * y or sum may be x or residual itself (same pointer and ld).
 */
flce_status_t ln_fwd(int kind, int dtype, const void* x, int64_t ld_x, const void* residual,
                     int64_t ld_residual, const void* weight, const void* bias, int param_dtype,
                     int64_t N, int64_t H, float eps, void* y, int64_t ld_y, void* sum,
                     int64_t ld_sum, float* mean, float* rstd, flce_stream_t stream);

/* Bytes of workspace ln_bwd needs; 0 for invalid sizes. */
size_t ln_workspace_size(int64_t N, int64_t H);

/*
 * ln_bwd
 *
 *  x             what ln_fwd normalised (`sum` where it had a residual).
 *  mean, rstd    fp32 [N], as ln_fwd wrote them (mean NULL for FLCE_NORM_RMS).
 *  grad_sum      [N, H] of `dtype` or NULL: the gradient that reaches `sum`
 *                from elsewhere (the residual stream), added to grad_x.
 *  grad_x        [N, H] of `dtype` output, or NULL to skip.
 *  grad_weight, grad_bias  fp32 [H] outputs, or NULL to skip.
 *  accumulate    0: grad_weight / grad_bias are overwritten; 1: added to.
 *  workspace     >= ln_workspace_size(N, H) bytes, 256-byte aligned; contents
 *                on entry are ignored.
 *
 * grad_x may be grad_y, grad_sum or x itself (same pointer and ld; with ld at
 * least H).  The sums over rows run in an order that the sizes and the layout
 * fix: the results are the same from run to run.  Their chains of fp32 additions
 * stay short: a call of very many rows makes several launches.
 */
flce_status_t ln_bwd(int kind, int dtype, const void* grad_y, int64_t ld_grad_y, const void* x,
                     int64_t ld_x, const void* weight, int param_dtype, const float* mean,
                     const float* rstd, const void* grad_sum, int64_t ld_grad_sum, int64_t N,
                     int64_t H, void* grad_x, int64_t ld_grad_x, float* grad_weight,
                     float* grad_bias, int accumulate, void* workspace, size_t workspace_bytes,
                     flce_stream_t stream);

/* ------------------------------------------------------------------------
 * The optimiser's step
 * ------------------------------------------------------------------------
 * The tables of tensors below are HOST memory and are read before the call
 * returns; the pointers in them are device pointers.
 */

/* A tensor of n contiguous elements (at most 2^41) of `dtype` (BF16, FP16 or FP32). */
typedef struct {
  const void* data;
  int64_t n;
  int32_t dtype;
  int32_t reserved; /* 0 */
} flce_tensor_t;

/* Bytes of workspace grad_norm needs for `count` tensors; 0 for count < 0. */
size_t grad_norm_workspace_size(int64_t count);

/*
 * grad_norm -- the 2-norm of many gradients together, and the factor for the
 * step that clips it:
 *     out[0] = norm  = |grad_scale| * sqrt(sum of all squares)
 *     out[1] = scale = grad_scale * min(1, max_norm / (norm + eps))
 *  or NaN as scale where the norm is not finite (adamw_step can then skip the
 *  step).  Squares are summed in fp32: a gradient above 1.8e19 in size makes
 *  the norm infinite, and squares of gradients below 1e-19 lose bits.
 *
 *  tensors, count  `count` >= 0 tensors; n = 0 is allowed.  All together, each
 *                  rounded up to 32 KB, less than 2^46 bytes.
 *  grad_scale      finite; what the gradients are to be multiplied by (1, or
 *                  the inverse of a loss scale).
 *  max_norm, eps   >= 0; max_norm infinity: no clipping.
 *  out             fp32 [2], device.
 *  workspace       >= grad_norm_workspace_size(count) bytes, 256-byte aligned;
 *                  contents on entry are ignored.
 *
 * The sum's order is fixed by the sizes: the same result from run to run.
 */
flce_status_t grad_norm(const flce_tensor_t* tensors, int64_t count, float grad_scale,
                        float max_norm, float eps, float* out, void* workspace,
                        size_t workspace_bytes, flce_stream_t stream);

/* Elements that share a scale in 8-bit moments. */
#define FLCE_ADAMW_BLOCK 256

/*
 * One tensor of an AdamW step: n contiguous elements each, at most 2^41.
 *  moment_bits  32: exp_avg and exp_avg_sq are fp32 [n], the scales NULL.
 *               8:  both are e4m3 numbers (1 byte) [n], and the scales fp32
 *                   [ceil(n / FLCE_ADAMW_BLOCK)]; element i of exp_avg stands
 *                   for number * scale[i / FLCE_ADAMW_BLOCK], element i of
 *                   exp_avg_sq for the square of that.
 *  copy         [n] of copy_dtype, or NULL: also gets the new parameter,
 *               rounded (the 16-bit weight that the products read).
 *  lr_scale     multiplies the step's lr for this tensor.
 * param and grad may each be BF16, FP16 or FP32.  No tensor of a call overlaps
 * another that the call writes.
 */
typedef struct {
  void* param;
  const void* grad;
  void* exp_avg;
  void* exp_avg_sq;
  float* exp_avg_scale;
  float* exp_avg_sq_scale;
  void* copy;
  int64_t n;
  float lr_scale;
  float weight_decay;
  int32_t param_dtype, grad_dtype, copy_dtype, moment_bits;
} flce_adamw_tensor_t;

/*
 * The step's numbers.
 *  step            t >= 1, this step's number (the first is 1); step_dev, when
 *                  not NULL, is a device int64 that holds it instead.
 *  lr_dev          device fp32 that holds lr, or NULL.
 *  grad_scale_dev  device fp32 that the gradients are multiplied by (out + 1 of
 *                  grad_norm), or NULL: grad_scale is that factor then.
 *  skip_nonfinite  1: when the factor is not finite, nothing is written.
 *  stochastic      1: 8-bit moments are rounded stochastically, by bits that
 *                  `seed`, the step, the tensor's place in the call's table
 *                  and the element's place in the tensor fix; 0: to nearest.
 */
typedef struct {
  double lr, beta1, beta2, eps;
  int64_t step;
  const int64_t* step_dev;
  const float* lr_dev;
  const float* grad_scale_dev;
  float grad_scale;
  int32_t skip_nonfinite;
  int32_t stochastic;
  int32_t reserved; /* 0 */
  uint64_t seed;
} flce_adamw_t;

/*
 * adamw_step -- one AdamW step (decoupled weight decay) over `count` tensors:
 *     g = grad * factor
 *     m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
 *     p = p (1 - lr weight_decay)
 *         - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 * in fp32, with lr the step's times the tensor's lr_scale; p is rounded to its
 * type once.  The update takes m and v before they are rounded to 8 bits.
 *
 * 8-bit moments: each block of FLCE_ADAMW_BLOCK elements (counted from the
 * tensor's start) has scale = its largest |m| (or sqrt v) * (1 / 448), at least
 * 2^-126 unless the block is 0, and holds m * (1 / scale) (or sqrt v) as e4m3
 * numbers, each of these operations rounded to fp32.  A root that is not 0 is
 * held as at least the smallest number, 2^-9, so that no step divides a moment
 * by a root that was rounded to 0.  A moment that is not finite is held as NaN
 * and leaves the rest of its block alone.
 *
 * betas in [0, 1), eps >= 0 (above 0, one below 2^-126 counts as 2^-126), lr
 * finite.  Needs no workspace.
 */
flce_status_t adamw_step(const flce_adamw_tensor_t* tensors, int64_t count,
                         const flce_adamw_t* numbers, flce_stream_t stream);

/* ------------------------------------------------------------------------
 * Losses of post-training on materialised logits
 * ------------------------------------------------------------------------
 * Each takes logits [N, V], rows of V contiguous elements `ld` elements apart,
 * and gives the loss and, unless grad_logits is NULL, its gradient on them.
 * With p = softmax(z) of a row z:
 *
 *  dtype         type of logits and grad_logits: FLCE_DTYPE_BF16, _FP16, _FP32.
 *  ld, ld_grad   >= V; N times either at most 2^58.
 *  grad_logits   [N, V] output, rows ld_grad apart; may be logits itself (with
 *                the same ld: the logits are consumed), else it overlaps nothing.
 *                What lies between two rows is not written.
 *  N, V          rows (>= 0, < 2^31) and columns (1 to 2^31 - 1).
 *  ignore_index  rows whose target it is take no part: loss 0, gradient 0.
 *  reduction     flce_reduction_t.
 *  grad_scale    multiplies every gradient; grad_out_none, fp32 of the losses'
 *                size or NULL, too, loss by loss (reduction NONE only).
 *  loss          fp32 output: one element for SUM and MEAN.
 *  workspace     256-byte aligned, of at least the stated size; contents on
 *                entry are ignored.
 *  status_dev    device status word, or NULL: then the workspace's first word
 *                holds this call's bits when it is done.
 *
 * Pointers need the alignment of their elements only.  Rows (pointer and ld)
 * that lie equally far from a 16-byte boundary in logits and grad_logits are the
 * fast case.  Arithmetic is fp32, with one rounding to the gradient's type; sums
 * over rows are fp64 in a fixed order: the results are the same from run to run.
 * Logits of -inf are columns of probability 0.  A row with NaN or +inf, or of
 * -inf alone, has a loss and gradients of NaN, and no other row has (but the
 * rows of its pair).  A row that takes no part, or whose weight is 0, gets zeros
 * whatever it holds.
 */

/*
 * The numbers of a policy loss.
 *  clip_low, clip_high  >= 0; the ratio is cut to [1 - clip_low, 1 + clip_high];
 *                       infinity: not cut on that side.
 *  kl_weight            finite, >= 0.
 *  temperature          1e-4 to 1e4: what the logits were divided by to sample.
 */
typedef struct {
  float clip_low, clip_high;
  float kl_weight;
  float temperature;
} flce_policy_t;

/* Bytes of workspace policy_fwd_bwd and distill_fwd_bwd need for N rows; 0 for
 * invalid sizes. */
size_t row_loss_workspace_size(int64_t N);

/*
 * policy_fwd_bwd -- the clipped policy loss of sampled tokens with a KL term:
 *     logp  = z_t / T - logsumexp(z / T),   t the row's target
 *     ratio = exp(logp - old_logp),   A the row's advantage
 *     loss  = row_weight * ( -min(ratio A, clip(ratio) A)
 *                            + kl_weight (exp(d) - 1 - d) ),  d = ref_logp - logp
 *  MEAN divides by the number of rows that take part (NaN if there is none),
 *  whatever their weights.  Where the cut ratio is taken the first term has no
 *  gradient.  A ratio that is not cut, or an exp(d), beyond the range of fp32
 *  makes its row's loss infinite and its gradients infinite or NaN; an advantage
 *  of 0 takes no ratio.
 *
 *  target        int64 [N]; one outside [0, V) that is not ignore_index sets
 *                FLCE_STATUS_BIT_TARGET_RANGE, and its row takes no part.
 *  advantage     fp32 [N].
 *  old_logp      fp32 [N], or NULL: the ratio is 1 and its gradient that of
 *                logp (the first update on fresh samples).
 *  ref_logp      fp32 [N], or NULL where kl_weight is 0.
 *  row_weight    fp32 [N], or NULL (1).
 *  loss          [N] for NONE.
 *  logp          fp32 [N] output or NULL; 0 for rows that take no part.
 */
flce_status_t policy_fwd_bwd(const void* logits, int dtype, int64_t ld, void* grad_logits,
                             int64_t ld_grad, const int64_t* target, const float* advantage,
                             const float* old_logp, const float* ref_logp, const float* row_weight,
                             int64_t N, int64_t V, const flce_policy_t* numbers,
                             int64_t ignore_index, int reduction, float grad_scale,
                             const float* grad_out_none, float* loss, float* logp,
                             void* workspace, size_t workspace_bytes, int32_t* status_dev,
                             flce_stream_t stream);

/* Largest length of a teacher's list. */
#define FLCE_DISTILL_MAX_TOP 1024

/* Types of ids. */
typedef enum { FLCE_INDEX_INT64 = 0, FLCE_INDEX_INT32 = 1 } flce_index_t;

/*
 * distill_fwd_bwd -- the distance from a teacher of which each row has the
 * largest logits:
 *     q    = softmax(values / T) over the row's list
 *     loss = row_weight * T^2 * sum_k q_k (ln q_k - ln p_k),   p = softmax(z / T)
 *  MEAN divides by the number of rows that have a list (NaN if there is none).
 *
 *  ids           [N, top] of index_type (flce_index_t): the list's columns, up to
 *                the first negative one.  A row whose first id is negative takes
 *                no part.  One of V or above sets FLCE_STATUS_BIT_TARGET_RANGE and
 *                is left out; a column that is named twice has both shares.
 *  values        [N, top] of value_dtype (any of the three types): the teacher's
 *                logits or log-probabilities.  -inf: no share; a list of -inf alone
 *                gives loss 0 and gradient 0; NaN or +inf: the row's loss is NaN.
 *  top           1 to FLCE_DISTILL_MAX_TOP.
 *  temperature   1e-4 to 1e4.
 *  row_weight    fp32 [N], or NULL (1).
 *  loss          [N] for NONE.
 */
flce_status_t distill_fwd_bwd(const void* logits, int dtype, int64_t ld, void* grad_logits,
                              int64_t ld_grad, const void* ids, int index_type,
                              const void* values, int value_dtype, int64_t top,
                              const float* row_weight, int64_t N, int64_t V, float temperature,
                              int reduction, float grad_scale, const float* grad_out_none,
                              float* loss, void* workspace, size_t workspace_bytes,
                              int32_t* status_dev, flce_stream_t stream);

typedef enum {
  FLCE_PREFERENCE_SIGMOID = 0,
  FLCE_PREFERENCE_HINGE = 1,
  FLCE_PREFERENCE_IPO = 2
} flce_preference_kind_t;

/*
 * The numbers of a preference loss.
 *  kind             flce_preference_kind_t.
 *  average          1: a sequence's log-probability is the mean over its tokens
 *                   that take part (0 without any), 0: their sum.
 *  beta             > 0, finite.
 *  label_smoothing  in [0, 1); SIGMOID only, else 0.
 *  margin           finite; SIGMOID and HINGE only, else 0.
 */
typedef struct {
  int32_t kind, average;
  float beta, label_smoothing, margin;
} flce_preference_t;

/* Bytes of workspace preference_fwd_bwd needs; 0 for invalid sizes. */
size_t preference_workspace_size(int64_t N, int64_t pairs);

/*
 * preference_fwd_bwd -- a loss over `pairs` pairs of sequences, the chosen one of
 * pair i being sequence i and the rejected one sequence pairs + i, by
 *     s_q = sum (or mean) of z_t - logsumexp(z) over the sequence's tokens
 *     x   = (s_chosen - ref_chosen) - (s_rejected - ref_rejected),  u = beta x - margin
 *     SIGMOID  -(1 - label_smoothing) ln sigmoid(u) - label_smoothing ln sigmoid(-u)
 *     HINGE    max(0, 1 - u)
 *     IPO      (x - 1 / (2 beta))^2
 *  MEAN divides by `pairs` (NaN if 0).
 *
 *  target        int64 [N], as in policy_fwd_bwd.
 *  offsets       int64 [2 pairs + 1], device, rising: sequence q has the rows
 *                from offsets[q] up to offsets[q + 1]; NULL: 2 pairs sequences of
 *                one length.  Rows of no sequence get gradients of 0.  Offsets
 *                that fall or leave [0, N] set FLCE_STATUS_BIT_SEQUENCE_RANGE, and
 *                sequences are then cut to what lies within.
 *  ref_logp      fp32 [2 pairs]: the reference model's s, or NULL (0).
 *  pairs         >= 0, < 2^30.
 *  grad_logits   as above; N * ceil(V / 1024) < 2^31 unless it is NULL.
 *  loss          [pairs] for NONE.
 *  logp          fp32 [2 pairs] output or NULL: s.
 */
flce_status_t preference_fwd_bwd(const void* logits, int dtype, int64_t ld, void* grad_logits,
                                 int64_t ld_grad, const int64_t* target, const int64_t* offsets,
                                 const float* ref_logp, int64_t pairs, int64_t N, int64_t V,
                                 const flce_preference_t* numbers, int64_t ignore_index,
                                 int reduction, float grad_scale, const float* grad_out_none,
                                 float* loss, float* logp, void* workspace,
                                 size_t workspace_bytes, int32_t* status_dev,
                                 flce_stream_t stream);

/* ------------------------------------------------------------------------
 * The table at the model's other end
 * ------------------------------------------------------------------------ */

/*
 * embedding_fwd -- y[n] = table[ids[n]] * scale, rounded once.
 *
 *  dtype         type of table and y: FLCE_DTYPE_BF16, _FP16 or _FP32.
 *  table         [V, H], rows ld_table (>= H) apart.
 *  ids           [N] of index_type (flce_index_t).  One outside [0, V) gives a
 *                row of zeros and sets FLCE_STATUS_BIT_TARGET_RANGE.
 *  N, V, H       N >= 0 (< 2^31), V 1 to 2^31 - 1, H 1 to 2^24 - 1.
 *  y             [N, H] output, rows ld_y (>= H) apart.
 *  status_dev    device status word, or NULL (not reported).
 */
flce_status_t embedding_fwd(int dtype, const void* table, int64_t ld_table, const void* ids,
                            int index_type, int64_t N, int64_t V, int64_t H, float scale, void* y,
                            int64_t ld_y, int32_t* status_dev, flce_stream_t stream);

/* Bytes of workspace embedding_bwd needs; 0 for sizes that it refuses. */
size_t embedding_workspace_size(int64_t N, int64_t V, int64_t H);

/*
 * embedding_bwd -- the table's gradient:
 *     grad_table[v] = scale * sum of grad_y[n] over the tokens n with ids[n] = v
 *
 *  dtype          type of grad_y [N, H], rows ld_grad_y (>= 0) apart.
 *  N, V, H        N < 2^31 - 32, V < 2^31 - 1, H <= 2097120, and
 *                 ceil(N / 32) * ceil(H / 128) <= 2^33 - 2^15 - 4.
 *  padding_index  tokens of this id add nothing; -1: none.
 *  grad_table     fp32 [V, H], contiguous.
 *  accumulate     0: every row is written (zeros where no token is); 1: added to,
 *                 and rows of no token are not touched (a shared weight's
 *                 gradient, as flce_fwd_bwd left it).
 *  workspace      >= embedding_workspace_size(...) bytes, 256-byte aligned;
 *                 contents on entry are ignored.
 *  status_dev     device status word, or NULL (not reported).
 *
 * An id outside [0, V) adds nothing and sets FLCE_STATUS_BIT_TARGET_RANGE.  Sums
 * are fp32 in an order that the ids and sizes fix: the same from run to run.
 */
flce_status_t embedding_bwd(int dtype, const void* grad_y, int64_t ld_grad_y, const void* ids,
                            int index_type, int64_t N, int64_t V, int64_t H, float scale,
                            int64_t padding_index, float* grad_table, int accumulate,
                            void* workspace, size_t workspace_bytes, int32_t* status_dev,
                            flce_stream_t stream);

/* ------------------------------------------------------------------------
 * Diagnostics (no counterpart on the pages)
 * ------------------------------------------------------------------------ */

/* Time limit of every pipeline wait inside the kernels, in nanoseconds of
 * %globaltimer (default 2e9).  Applies to calls enqueued afterwards. */
void flce_set_wait_timeout_ns(uint64_t timeout_ns);

/* Enqueues a kernel whose pipeline wait can never be satisfied: after
 * timeout_ns it must give up, set FLCE_STATUS_BIT_TIMEOUT in *status_dev and
 * return.  Checks the failure path of the bounded waits without faulting. */
flce_status_t flce_selftest_wait_timeout(int32_t* status_dev, uint64_t timeout_ns,
                                         flce_stream_t stream);

/* Kernel timing: while enabled, every kernel the library enqueues is
 * bracketed by a pair of CUDA events on its stream (the library creates up
 * to `capacity` pairs once).  flce_profile_read synchronises on the recorded
 * events and returns, for each recorded launch, its kernel id (below) and
 * duration in ms; returns the number written (<= max).  Not thread-safe. */
enum {
  FLCE_KERNEL_COUNT_TARGETS = 0,
  FLCE_KERNEL_GEMM_FWD = 1,
  FLCE_KERNEL_ROW_FINALIZE = 2,
  FLCE_KERNEL_GRAD_LOGITS = 3,
  FLCE_KERNEL_GEMM_BWD = 4,
  FLCE_KERNEL_LOSS_REDUCE = 5,
  FLCE_KERNEL_CE_ROWS = 6,
  FLCE_KERNEL_ZERO = 7,
  FLCE_KERNEL_BIAS_REDUCE = 8,
  FLCE_KERNEL_GH_REDUCE = 9,
  FLCE_KERNEL_LN_FWD = 10,
  FLCE_KERNEL_LN_BWD = 11,
  FLCE_KERNEL_LN_REDUCE = 12,
  FLCE_KERNEL_GRAD_NORM = 13,
  FLCE_KERNEL_ADAMW = 14,
  FLCE_KERNEL_ROW_LOSS = 15,   /* policy, distill, and the row statistics of a preference loss */
  FLCE_KERNEL_ROW_COUNT = 16,
  FLCE_KERNEL_PAIR_LOSS = 17,
  FLCE_KERNEL_ROW_GRAD = 18,
  FLCE_KERNEL_EMBEDDING = 19,
  FLCE_KERNEL_TOKEN_SORT = 20,
  FLCE_KERNEL_EMBEDDING_BWD = 21,
  FLCE_KERNEL_EMBEDDING_JOIN = 22
};
const char* flce_kernel_name(int kernel_id);
flce_status_t flce_profile_enable(int capacity);
void flce_profile_disable(void);
int flce_profile_read(int* kernel_ids, float* ms, int max);

#ifdef __cplusplus
}
#endif
#endif /* FLCE_H_ */
