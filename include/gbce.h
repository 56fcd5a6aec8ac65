/*
 * gbce.h -- C ABI of libgbce.so: row-wise log-softmax and token cross-entropy
 * over a [rows, vocab] logit matrix on one NVIDIA GB300 (sm_103a).
 *
 * What is computed (z_j = x_j / T for a row x of length V, temperature T):
 *
 *   log p_t = -softplus( log sum_{j != t} exp(z_j - m_t) + m_t - z_t ),
 *   m_t     = max_{j != t} z_j,   softplus(a) = max(a,0) + log1p(exp(-|a|)),
 *
 * which equals z_t - logsumexp_j z_j but never rounds to exactly 0 (and is
 * never positive) when the target leads the other logits by a wide margin.
 * This is the collapse-safe form of "Fix softmax collapse in CE, GRPO,
 * KL/JSD and softmax" (Liger-Kernel PR #1555), section "Summary": the first
 * pass also accumulates the sum without the target, and the loss is
 * softplus(log(sum_others) + m - x_y).
 *
 * Conventions shared by every entry point:
 *
 *  - Memory.  Every pointer argument is DEVICE memory owned by the caller,
 *    except that `stream` is a cudaStream_t handle (NULL = legacy default
 *    stream).  The library allocates nothing, frees nothing and keeps no
 *    state between calls; scratch space is the caller's `workspace`.
 *  - Layout.  Logits are row-major: row r starts `r * row_stride` ELEMENTS
 *    after `logits`, and its first `vocab` elements are used.  row_stride >=
 *    vocab.  Index, label, mask and per-row outputs are dense.  The logits
 *    pointer must be aligned to its element size; rows need not be 16-byte
 *    aligned (a misaligned head/tail is read with scalar loads).
 *  - Types.  Logits are fp32 or bf16; every computation is fp32; log-probs,
 *    losses and log-sum-exps are written as fp32; dlogits have the logits'
 *    type (bf16 rounded to nearest even).
 *  - Accuracy.  Against an fp64 evaluation of the same definitions: log-probs,
 *    losses and entropies within 1e-5 to 2e-5 relative; dlogits within 2e-5
 *    (fp32) or 4e-3 (bf16) relative per row.  Confident rows keep these
 *    bounds (the sums run over the non-target columns, the target gradient
 *    is expm1(log p)), down to fp32's subnormals.  A value fp32 cannot hold
 *    at all, such as a log p of -1e-50, is written as 0.  Soft-capped logits
 *    carry the fp32 rounding of cap * tanh(x / cap) in every exponent.  A
 *    backward call takes the forward's fp32 log p and entropy as they are.
 *  - Masked columns and NaN.  A logit of -inf, or one so far below (x / T under
 *    -1.48e9, the type's lowest value for one) that no shift can be taken off it,
 *    has no mass beside any other.  Except in the losses of post-training, a row
 *    that holds nothing else (and is not all -inf) can be NaN; under -2.98e9 it is.  A NaN logit makes its
 *    row's outputs NaN, and no other row's.
 *  - Asynchrony.  Every call only enqueues work on `stream` and returns; it
 *    never synchronizes the host.  The returned status reports HOST-side
 *    argument checks (and launch errors) only.  Some kernels of a call are
 *    programmatic dependents of the kernel before them on the stream (their
 *    launch overlaps it), and each waits for that kernel to complete before
 *    its first global memory access; to the caller a call still runs in
 *    stream order, after all earlier work on `stream` and before all later
 *    work.
 *  - Device-side errors.  A label or index outside [0, vocab) (labels equal
 *    to ignore_index excepted) sets a bit in `*dev_status` (atomic OR; pass
 *    NULL to skip reporting) and makes that row's outputs NaN.  A pipeline
 *    wait that exceeds its time limit sets GBCE_DEV_TIMEOUT and the kernel
 *    returns instead of hanging.  Nothing traps.  The caller zeroes
 *    *dev_status and reads it whenever it likes.
 *  - Threading.  Calls on different streams may run concurrently provided
 *    their output and workspace buffers do not overlap.
 */
#ifndef GBCE_H
#define GBCE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GBCE_OK = 0,
    GBCE_EINVAL = 1,     /* null pointer, bad size/stride/temperature, aliasing */
    GBCE_EDTYPE = 2,     /* unsupported dtype or misaligned element pointer */
    GBCE_ECUDA = 3,      /* a CUDA launch or attribute call failed */
    GBCE_EWORKSPACE = 4  /* workspace smaller than gbce_workspace_size() */
} gbce_status;

typedef enum { GBCE_F32 = 0, GBCE_BF16 = 1 } gbce_dtype;

typedef enum { GBCE_NONE = 0, GBCE_SUM = 1, GBCE_MEAN = 2 } gbce_reduction;

/* Bits OR-ed into *dev_status by the kernels. */
#define GBCE_DEV_BAD_LABEL 1   /* a label outside [0, vocab) and != ignore_index */
#define GBCE_DEV_BAD_INDEX 2   /* a gather index outside [0, vocab) */
#define GBCE_DEV_TIMEOUT 4     /* a pipeline wait gave up; outputs of that row are invalid */

/* Largest number of gathered indices per row that selective_logsoftmax takes. */
#define GBCE_MAX_K 16

/*
 * Bytes of workspace that any call on a [rows, vocab] problem with k indices
 * per row needs (k = 1 for the cross-entropy calls).  A pure function of its
 * arguments: no CUDA call, valid for any device.  Returns 0 for rows <= 0.
 */
size_t gbce_workspace_size(int64_t rows, int64_t vocab, int64_t k);

/* Static, human-readable name of a status code. */
const char *gbce_status_string(gbce_status status);

/*
 * Number of kernels this library has enqueued in this process so far (all
 * devices, all streams), for accounting in benchmarks.  Thread-safe.
 */
uint64_t gbce_kernel_launches(void);

/*
 * Selective log-softmax: logp_out[r, k] = log p_{index[r, k]} of row r at
 * temperature T, for rows with row_mask[r] != 0 (or all rows when row_mask
 * is NULL); masked-out rows are not read and get 0.  With entropy_out, the
 * same sweep also gives the entropy of each row's softmax,
 * entropy_out[r] = -sum_j p_j log p_j (0 log 0 = 0; 0 for masked rows),
 * with the dominant column's 1 - p taken from its accurate log p, so a
 * confident row keeps its small positive entropy whichever column it is
 * confident in (when that is not the first index, the row's entropy is
 * recomputed around it in a second pass over that row).
 *
 * Source: "perf(rlhf): chunk selective_log_softmax instead of looping per
 * token" (ms-swift PR #10337), "PR information": the naive
 * gather(logits.log_softmax(-1)) with top-K indices, temperature and a row
 * mask, here in one launch over all rows; accurate log-probs as in "Fix
 * softmax collapse ..." (Liger-Kernel PR #1555), "Summary", second bullet;
 * the entropy taking the others' sum from the same term as the target's
 * log p: the unsloth-zoo #2080 commit quoted there, "Fix", forward bullet.
 *
 *   logits     [rows, row_stride] fp32/bf16
 *   index      [rows, k] int64, 1 <= k <= GBCE_MAX_K; duplicates allowed
 *   row_mask   [rows] uint8 or NULL
 *   logp_out   [rows, k] fp32
 *   entropy_out [rows] fp32 or NULL (NULL: the sweep skips the entropy)
 *   workspace  >= gbce_workspace_size(rows, vocab, k) bytes (may be NULL
 *              when that size is 0), 16-byte aligned
 * Errors: GBCE_EINVAL for NULL logits/index/logp_out with rows > 0,
 * vocab < 1, row_stride < vocab, k outside [1, GBCE_MAX_K], temperature not
 * finite and > 0; GBCE_EDTYPE; GBCE_EWORKSPACE.  Out-of-range indices of
 * live rows: GBCE_DEV_BAD_INDEX and a NaN output for that (r, k); the
 * entropy of a row whose first index is out of range is NaN.
 */
gbce_status selective_logsoftmax(const void *logits, gbce_dtype dtype, int64_t rows,
                                 int64_t vocab, int64_t row_stride, const int64_t *index,
                                 int64_t k, float temperature, const uint8_t *row_mask,
                                 float *logp_out, float *entropy_out, void *workspace,
                                 size_t workspace_bytes, int32_t *dev_status, void *stream);

/*
 * Selective log-softmax backward: the gradient of sum_k g[r, k] *
 * log p_{index[r, k]} with respect to the logits,
 *   dlogits[r, j] = (1/T) * ( sum_{k : index[r, k] = j} g[r, k] - G_r * p_j ),
 * G_r = sum_k g[r, k], with every gathered column t evaluated as
 *   (1/T) * ( -g_t * expm1(log p_t) - (G_r - g_t) * exp(log p_t) )
 * (g_t = the upstream of every k that gathers t) so that 1 - p_t keeps its
 * value when p_t rounds to 1; masked-out rows get a zero row.  With
 * grad_entropy, the gradient of gH_r * H_r (H_r the row entropy of the
 * forward's entropy_out) is added:
 *   - (gH_r / T) * p_j * (log p_j + H_r)   for every column j,
 * 0 where p_j = 0, with log p of the gathered columns from saved_logp.  The
 * other columns' p_j are taken relative to index[r, 0]; a row with
 * saved_logp[r, 0] < -40 reads its max and sum in a second pass over that
 * row and takes them relative to the max (hundreds of nats between the
 * two would cost fp32 accuracy).
 *
 * Source: the gradient a GRPO-style loss sends back through the accurate
 * log-probs of "Fix softmax collapse in CE, GRPO, KL/JSD and softmax"
 * (Liger-Kernel PR #1555), "Summary", second bullet (-expm1(logp) for
 * 1 - p_y); gradients are part of the checked behaviour of "perf(rlhf):
 * chunk selective_log_softmax instead of looping per token", "PR
 * information".
 *
 *   index       [rows, k] int64, as given to selective_logsoftmax
 *   row_mask    [rows] uint8 or NULL
 *   grad_logp   [rows, k] fp32, device: dL/d logp_out
 *   saved_logp  [rows, k] fp32: selective_logsoftmax's output for the same
 *               logits, index and temperature
 *   grad_entropy  [rows] fp32 or NULL: dL/d entropy_out
 *   saved_entropy [rows] fp32: the forward's entropy_out; NULL exactly when
 *               grad_entropy is NULL
 *   dlogits     [rows, dlogits_row_stride], the logits' dtype; must not
 *               overlap the logits
 * Errors: as ce_bwd; a row with an index outside [0, vocab) sets
 * GBCE_DEV_BAD_INDEX and gets a NaN row.
 */
gbce_status selective_logsoftmax_bwd(const void *logits, gbce_dtype dtype, int64_t rows,
                                     int64_t vocab, int64_t row_stride, const int64_t *index,
                                     int64_t k, float temperature, const uint8_t *row_mask,
                                     const float *grad_logp, const float *saved_logp,
                                     const float *grad_entropy, const float *saved_entropy,
                                     void *dlogits, int64_t dlogits_row_stride,
                                     int32_t *dev_status, void *stream);

/*
 * Options of the token cross-entropy calls (ce_fwd, ce_bwd,
 * ce_fwd_bwd_fused).  A NULL pointer means all defaults (plain CE).
 *
 *   label_smoothing  eps in [0, 1]: the target distribution puts 1 - eps on
 *                    the label and eps / vocab on every class, so a kept
 *                    row's loss is (1 - eps)(-log p_y) + eps * mean_j(-log p_j)
 *                    and its gradient (g/T)(p_j - (1 - eps)[j == y] - eps/vocab),
 *                    the label column in the expm1(log p_y) form ("Fix
 *                    softmax collapse ...", the unsloth-zoo #2080 commit's
 *                    "Fix", backward bullet).  A row with a -inf logit has
 *                    an infinite smoothed loss, as the definition gives.
 *   dft              nonzero: weight each kept row's loss and gradient by its
 *                    own p_y, held constant in the backward (the DFT loss
 *                    -p_y log p_y of ms-swift PR #10353, "PR information").
 *                    Combines with label_smoothing (the weight multiplies
 *                    the smoothed row loss).
 *   softcap          cap >= 0 (0: off): every logit x becomes cap * tanh(x / cap)
 *                    before the temperature and the softmax; the gradient
 *                    with respect to x takes the factor 1 - tanh^2(x / cap).
 *                    Its tanh per element makes these calls ALU-bound, and
 *                    the fused call then runs as a statistics pass and a
 *                    gradient pass.  Logit soft-capping is named among the
 *                    options of the fused losses on "Fix softmax collapse
 *                    ..." (the unsloth-zoo #2080 commit, "Accuracy" tests).
 * ce_bwd must be given the same options as the ce_fwd whose log p it takes.
 * An eps outside [0, 1] (or NaN), or a negative or non-finite softcap, makes
 * the call return GBCE_EINVAL before any GPU work.
 */
typedef struct gbce_ce_options {
    float label_smoothing;
    int32_t dft;
    float softcap;
} gbce_ce_options;

/*
 * Token cross-entropy forward.  For rows whose label is not ignore_index:
 * loss_r = -log p_{labels[r]} at temperature T; ignored rows are skipped
 * before any read of their logits and get loss 0.
 *
 * Source: "Fix softmax collapse ..." (Liger-Kernel PR #1555), "Summary",
 * first bullet (loss = softplus(log(sum_others) + m - x_y)); row selection
 * before any vocabulary work from ms-swift PR #10353, "PR information".
 *
 *   labels      [rows] int64
 *   options     gbce_ce_options or NULL (plain CE)
 *   reduction   GBCE_NONE: loss_out[rows] = loss_r;
 *               GBCE_SUM:  loss_out[0] = sum_r loss_r;
 *               GBCE_MEAN: loss_out[0] = sum_r loss_r / n_items, 0 when
 *               n_items == 0 (all rows ignored).
 *   logp_out    [rows] fp32 or NULL: log p of the label (0 when ignored);
 *               ce_bwd takes it back as saved_logp.
 *   lse_out     [rows] fp32 or NULL: logsumexp_j z_j (0 when ignored).
 *   n_items_out [1] int64 or NULL: number of rows with label != ignore_index.
 *   workspace   >= gbce_workspace_size(rows, vocab, 1) bytes.
 * Sums are deterministic (fixed order) and taken in fp64.
 * Errors: as selective_logsoftmax; bad labels set GBCE_DEV_BAD_LABEL and
 * give NaN for that row (and hence a NaN sum/mean).
 */
gbce_status ce_fwd(const void *logits, gbce_dtype dtype, int64_t rows, int64_t vocab,
                   int64_t row_stride, const int64_t *labels, int64_t ignore_index,
                   float temperature, gbce_reduction reduction,
                   const gbce_ce_options *options, float *loss_out,
                   float *logp_out, float *lse_out, int64_t *n_items_out, void *workspace,
                   size_t workspace_bytes, int32_t *dev_status, void *stream);

/*
 * Token cross-entropy backward from saved statistics:
 *   dlogits[r, j] = (g_r / T) * exp(z_j - z_y + log p_y)   for j != y,
 *   dlogits[r, y] = (g_r / T) * expm1(log p_y),
 * i.e. g_r * (softmax - onehot) / T with the target term in the form that
 * does not round to zero (with options: the smoothed and DFT-weighted
 * gradient described at gbce_ce_options); ignored rows get a zero row.  A
 * row with log p_y < -40 evaluates its exponents from the row's max instead
 * (z_j - z_max - log S), read in a second pass over that row: taken
 * relative to the label, a column hundreds of nats above it would lose fp32
 * accuracy.  g_r = grad_out[r]
 * (NONE), grad_out[0] (SUM) or grad_out[0] / n_items (MEAN, 0 when
 * n_items == 0).
 *
 * Source: ms-swift PR #10353, "PR information", second bullet (backward
 * computed directly as g*softmax - g*onehot, zero weight for ignored
 * labels, a separate gradient buffer); the target term -expm1(log p_t) from
 * the unsloth-zoo #2080 commit quoted on "Fix softmax collapse ..."
 * (section "Fix", backward bullet).
 *
 *   grad_out    [rows] (NONE) or [1] fp32, device
 *   saved_logp  [rows] fp32 from ce_fwd's logp_out (same logits, labels, T)
 *   n_items     [1] int64 from ce_fwd; required for GBCE_MEAN, else ignored
 *   dlogits     [rows, dlogits_row_stride] of the logits' dtype; must not
 *               overlap the logits; dlogits_row_stride >= vocab
 * Errors: GBCE_EINVAL for NULL required pointers, overlap, bad strides or
 * temperature; bad labels set GBCE_DEV_BAD_LABEL and give a NaN row.
 */
gbce_status ce_bwd(const void *logits, gbce_dtype dtype, int64_t rows, int64_t vocab,
                   int64_t row_stride, const int64_t *labels, int64_t ignore_index,
                   float temperature, gbce_reduction reduction,
                   const gbce_ce_options *options, const float *grad_out,
                   const float *saved_logp, const int64_t *n_items, void *dlogits,
                   int64_t dlogits_row_stride, int32_t *dev_status, void *stream);

/*
 * Cross-entropy forward and backward in one call: the outputs of ce_fwd
 * and, with the upstream gradient known in advance, those of ce_bwd.  Each
 * row's logits are read from HBM once; the gradient pass re-reads them from
 * on-chip memory or L2.
 *
 * Source: as ce_fwd and ce_bwd; taking the gradient in the forward when the
 * upstream gradient is known follows the fused losses described in the
 * unsloth-zoo #2079 commit on "Fix softmax collapse ..." ("Summary").
 *
 * Arguments as in ce_fwd and ce_bwd; loss_out, dlogits and grad_out are
 * required, logp_out / lse_out / n_items_out are optional.
 */
gbce_status ce_fwd_bwd_fused(const void *logits, gbce_dtype dtype, int64_t rows,
                             int64_t vocab, int64_t row_stride, const int64_t *labels,
                             int64_t ignore_index, float temperature,
                             gbce_reduction reduction, const gbce_ce_options *options,
                             const float *grad_out, float *loss_out,
                             float *logp_out, float *lse_out, int64_t *n_items_out,
                             void *dlogits, int64_t dlogits_row_stride, void *workspace,
                             size_t workspace_bytes, int32_t *dev_status, void *stream);

/*
 * Vocabulary-parallel selective log-softmax: the vocabulary is split into
 * slices (e.g. one per device, as a vocab-parallel LM head leaves it), each
 * slice's statistics are computed where its logits are, the caller gathers
 * them (any transport: an all-gather over devices, or nothing when every
 * slice is on one device), and one combine gives the log-probs.  The
 * gradient is then computed slice by slice from the combined log-probs.
 * Token cross-entropy is the case k = 1, index = labels, ignore_index = the
 * ignored label: loss_r = -logp[r], and its gradient is vocab_slice_grad
 * with grad_logp[r] = -(upstream of row r).
 *
 * Source: "Fix softmax collapse in CE, GRPO, KL/JSD and softmax"
 * (Liger-Kernel PR #1555), "Summary", first bullet: the vocab-parallel form
 * keeps, per slice, the sum over the columns other than the target, and
 * reduces both sums across slices.
 *
 * Slices are described by their global column ranges: slice i holds columns
 * [slice_offsets[i], slice_offsets[i + 1]) of a vocabulary of `vocab`
 * columns, slice_offsets[0] = 0 and slice_offsets[slices] = vocab.
 * Indices are global columns.  A row is skipped (log p 0, zero gradient)
 * when row_mask[r] == 0 or index[r, 0] == ignore_index.  Label smoothing,
 * DFT, soft-capping and the entropy are not available on this path.
 */
#define GBCE_MAX_SLICES 64

/*
 * Statistics of one slice.  logits: [rows, row_stride] holding the slice's
 * slice_vocab columns, global columns [vocab_offset, vocab_offset +
 * slice_vocab).  partials: [rows, 2 + k] fp32, device, written as
 *   partials[r, 0] = m_r = max over the slice's non-target columns of x / T
 *                    (in units of x, i.e. the raw max),
 *   partials[r, 1] = sum of exp((x_j - m_r) / T) over those columns,
 *   partials[r, 2 + k'] = logit of index[r, k'] if this slice holds it, else 0;
 * a skipped row gets (-inf, 0, 0, ...).
 * Errors: as selective_logsoftmax; GBCE_EINVAL also for vocab_offset < 0 or
 * vocab_offset + slice_vocab > vocab.  Indices outside [0, vocab) are
 * reported by the combine.
 */
gbce_status vocab_slice_stats(const void *logits, gbce_dtype dtype, int64_t rows,
                              int64_t slice_vocab, int64_t row_stride, int64_t vocab_offset,
                              int64_t vocab, const int64_t *index, int64_t k,
                              int64_t ignore_index, const uint8_t *row_mask, float temperature,
                              float *partials, int32_t *dev_status, void *stream);

/*
 * Combine of all slices' partials, stacked in slice order as
 * partials[slices, rows, 2 + k] (device).  slice_offsets: HOST array of
 * slices + 1 int64 (read during the call).  logp_out: [rows, k] fp32 as
 * selective_logsoftmax would give on the whole vocabulary (a bad index: NaN
 * and GBCE_DEV_BAD_INDEX); target_logit_out: [rows] fp32 or NULL, the logit
 * of index[r, 0], which vocab_slice_grad needs; row_state_out: [rows, 2]
 * fp32 or NULL, each row's max M over all its columns (raw logit) and S =
 * sum_j exp((x_j - M) / T) (a skipped row: -inf, 0), which vocab_slice_grad
 * takes for rows far below their max.  The merge runs in slice
 * order, so the result does not depend on the order the slices were
 * computed in.
 * Errors: GBCE_EINVAL for slices outside [1, GBCE_MAX_SLICES], offsets not
 * starting at 0 or not increasing, k outside [1, GBCE_MAX_K], a bad
 * temperature or NULL required pointers.
 */
gbce_status vocab_slice_combine(const float *partials, int64_t slices,
                                const int64_t *slice_offsets, int64_t rows, const int64_t *index,
                                int64_t k, int64_t ignore_index, const uint8_t *row_mask,
                                float temperature, float *logp_out, float *target_logit_out,
                                float *row_state_out, int32_t *dev_status, void *stream);

/*
 * Gradient of sum_k grad_logp[r, k] * logp[r, k] with respect to one
 * slice's logits (the columns of selective_logsoftmax_bwd that the slice
 * holds), from the combined log-probs and target logit:
 *   dlogits[r, j] = (1/T) (sum_{k : index[r, k] = j} g[r, k] - G_r p_j),
 *   p_j = exp((x_j - x_{t0}) / T + logp[r, 0]),
 * gathered columns in the -expm1 form.  A row with logp[r, 0] < -40 and a
 * row_state takes p_j = exp((x_j - M) / T) / S from the row state instead:
 * taken relative to index 0, a column hundreds of nats above it would lose
 * fp32 accuracy.
 *   logp         [rows, k] fp32 from vocab_slice_combine
 *   target_logit [rows] fp32 from vocab_slice_combine
 *   row_state    [rows, 2] fp32 from vocab_slice_combine, or NULL
 *   dlogits      [rows, dlogits_row_stride] of the logits' type, the slice's
 *                columns; must not overlap the logits
 * Errors: as selective_logsoftmax_bwd; a row with an index outside
 * [0, vocab) gets a NaN row and GBCE_DEV_BAD_INDEX.
 */
gbce_status vocab_slice_grad(const void *logits, gbce_dtype dtype, int64_t rows,
                             int64_t slice_vocab, int64_t row_stride, int64_t vocab_offset,
                             int64_t vocab, const int64_t *index, int64_t k, int64_t ignore_index,
                             const uint8_t *row_mask, float temperature, const float *grad_logp,
                             const float *logp, const float *target_logit,
                             const float *row_state, void *dlogits, int64_t dlogits_row_stride,
                             int32_t *dev_status, void *stream);

/*
 * The calls that start from hidden states: the logits are
 *   logits[r, v] = sum_d hidden[r, d] weight[v, d]
 * (the language-model head).  They are formed tile by tile and not kept: the
 * gradients form them again, a piece of the vocabulary at a time, and hold
 * that piece's gradient (in the inputs' type).  Only a fused call whose fp32
 * logits take at most 256 MB keeps them in its workspace instead of forming
 * them twice.  Log-probs, losses and gradients are those of the calls above on these
 * logits, the gradients with respect to hidden and weight:
 *   dhidden = dlogits . weight          dweight = dlogits^T . hidden.
 *
 * Source: the operators "softmax cross-entropy / selective log-softmax
 * behind a linear head" that the unsloth-zoo #2080 commit quoted on "Fix
 * softmax collapse ..." describes ("Fix": the running sum excludes the
 * target, log p_t = -softplus(log s_others + m - z_t), the target's gradient
 * by -expm1(log p_t)), row selection before any vocabulary work from
 * ms-swift PR #10353, "PR information".
 *
 *  - Types.  hidden, weight and their gradients have one type, fp32 or bf16.
 *    Products are summed in fp32; log-probs, losses and row states are fp32.
 *    In a bf16 call the gradient of the logits is rounded once to bf16
 *    (as ce_bwd returns it) before the products that give dhidden and
 *    dweight, which are summed in fp32 and rounded once: 1.7e-3 to 2.4e-3
 *    in norm against 64 bits, 1.66e-3 of it the gradients' own rounding.
 *  - Layout.  hidden: [rows, dim], weight: [vocab, dim], rows hidden_row_stride
 *    and weight_row_stride elements apart (>= dim), any alignment of the
 *    element type; likewise dhidden and dweight.  A bf16 weight whose rows
 *    start on 16 bytes is read in place; any other, and the live rows of
 *    hidden, are laid out anew in the workspace (a bf16 forward of up to 128
 *    such rows reads hidden in place too).
 *  - Rows left out (row_mask[r] == 0, or label == ignore_index) have no part
 *    in anything, whatever they hold (NaN included): log p 0, loss 0, row
 *    state (-inf, 0), dhidden 0, nothing in dweight.  Calls with gradients and
 *    longer forwards do no work for them; a bf16 forward of up to 128 rows
 *    may read them all the same, and drops what it made.
 *  - A label outside [0, vocab), or in the backward an index outside it,
 *    sets its dev_status bit, makes the row's log p, loss and dhidden NaN
 *    and leaves the row out of dweight.  In the selective forward an index
 *    outside [0, vocab) makes its own log p NaN only.
 *  - Row state.  row_state[r] = (M, S): the max of the row's logits and
 *    sum_v exp((z_v - M) / T), as vocab_slice_combine gives it.  A backward
 *    call takes it with the forward's log p; it forms the logits again, by
 *    the same steps.
 *  - dweight with accumulate != 0: dweight += the gradient (read, added in
 *    fp32, rounded once), else dweight = the gradient, rows of the table
 *    that get none being zeros.  dhidden or dweight may be NULL: it is not
 *    computed.
 *  - workspace: gbce_linear_workspace_size bytes, 32-byte aligned, of one
 *    call at a time (a captured graph keeps its own).
 *  - Sums are in a fixed order: the same call gives the same bits.
 *  - A pipeline wait that gives up sets GBCE_DEV_TIMEOUT; the call's outputs
 *    are then invalid.
 * Errors: GBCE_EINVAL for rows outside [0, 2^24], dim outside [1, 2^20],
 * vocab < 1, strides below dim, k, temperature and NULL pointers as above,
 * outputs that overlap an input or each other, no gradient wanted at all
 * (a call without rows is refused for the same, but takes NULL for its empty
 * inputs; a dhidden that is wanted has an address there too); GBCE_EDTYPE;
 * GBCE_EWORKSPACE.  Label smoothing, DFT, soft-capping and the entropy are not
 * available on this path.
 */

/* Bytes of workspace of a call; backward: 0 for the two forward calls.
 * A pure function of its arguments; 0 for arguments that no call takes. */
size_t gbce_linear_workspace_size(int64_t rows, int64_t vocab, int64_t dim, int64_t k,
                                  gbce_dtype dtype, int backward);

/* selective_logsoftmax of hidden . weight^T.  row_state_out: [rows, 2] or NULL. */
gbce_status linear_selective_logsoftmax(const void *hidden, int64_t hidden_row_stride,
                                        const void *weight, int64_t weight_row_stride,
                                        gbce_dtype dtype, int64_t rows, int64_t vocab, int64_t dim,
                                        const int64_t *index, int64_t k, float temperature,
                                        const uint8_t *row_mask, float *logp_out,
                                        float *row_state_out, void *workspace,
                                        size_t workspace_bytes, int32_t *dev_status, void *stream);

/* Gradient of sum_k grad_logp[r, k] * logp[r, k] with respect to hidden and
 * weight.  grad_logp, saved_logp: [rows, k]; row_state: [rows, 2]. */
gbce_status linear_selective_logsoftmax_bwd(
    const void *hidden, int64_t hidden_row_stride, const void *weight, int64_t weight_row_stride,
    gbce_dtype dtype, int64_t rows, int64_t vocab, int64_t dim, const int64_t *index, int64_t k,
    float temperature, const uint8_t *row_mask, const float *grad_logp, const float *saved_logp,
    const float *row_state, void *dhidden, int64_t dhidden_row_stride, void *dweight,
    int64_t dweight_row_stride, int accumulate, void *workspace, size_t workspace_bytes,
    int32_t *dev_status, void *stream);

/* ce_fwd of hidden . weight^T; logp_out, row_state_out and n_items_out may be NULL. */
gbce_status linear_ce_fwd(const void *hidden, int64_t hidden_row_stride, const void *weight,
                          int64_t weight_row_stride, gbce_dtype dtype, int64_t rows, int64_t vocab,
                          int64_t dim, const int64_t *labels, int64_t ignore_index,
                          float temperature, gbce_reduction reduction, float *loss_out,
                          float *logp_out, float *row_state_out, int64_t *n_items_out,
                          void *workspace, size_t workspace_bytes, int32_t *dev_status,
                          void *stream);

/* Both gradients from linear_ce_fwd's log p and row state; grad_out and
 * n_items as in ce_bwd. */
gbce_status linear_ce_bwd(const void *hidden, int64_t hidden_row_stride, const void *weight,
                          int64_t weight_row_stride, gbce_dtype dtype, int64_t rows, int64_t vocab,
                          int64_t dim, const int64_t *labels, int64_t ignore_index,
                          float temperature, gbce_reduction reduction, const float *grad_out,
                          const float *saved_logp, const float *row_state, const int64_t *n_items,
                          void *dhidden, int64_t dhidden_row_stride, void *dweight,
                          int64_t dweight_row_stride, int accumulate, void *workspace,
                          size_t workspace_bytes, int32_t *dev_status, void *stream);

/* Loss and both gradients in one call. */
gbce_status linear_ce_fwd_bwd_fused(
    const void *hidden, int64_t hidden_row_stride, const void *weight, int64_t weight_row_stride,
    gbce_dtype dtype, int64_t rows, int64_t vocab, int64_t dim, const int64_t *labels,
    int64_t ignore_index, float temperature, gbce_reduction reduction, const float *grad_out,
    float *loss_out, float *logp_out, float *row_state_out, int64_t *n_items_out, void *dhidden,
    int64_t dhidden_row_stride, void *dweight, int64_t dweight_row_stride, int accumulate,
    void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream);

/*
 * The table's other end: rows of a [vocab, dim] table by token, times a
 * scale (with a tied table, the weight of the calls above), and the
 * gradient of that lookup, which with accumulate joins the head's gradient
 * of the same table:
 *   out[r]    = scale * table[tokens[r]]
 *   dtable[v] = scale * sum_{r : tokens[r] = v} grad_out[r]   (+ dtable[v])
 * summed in fp32 in a fixed order and rounded once.  tokens: [rows] int64; a
 * token equal to ignore_index (padding) gives a row of zeros and no
 * gradient, whatever its gradient row holds; one outside [0, vocab)
 * otherwise sets GBCE_DEV_BAD_INDEX, gives a NaN row and no gradient.
 * Without accumulate every row of dtable is written (zeros where no token
 * names it); with it only the rows that tokens name are touched.  One type
 * for table, out, grad_out and dtable; any row strides >= dim, any alignment
 * of the element type; outputs must not overlap inputs; scale finite.
 * workspace: gbce_embedding_workspace_size bytes, 16-byte aligned.
 *
 * Source: no page has it; it completes the gradient of a tied head (above).
 */
size_t gbce_embedding_workspace_size(int64_t rows, int64_t vocab, int64_t dim);

gbce_status embedding_lookup(const void *table, int64_t table_row_stride, gbce_dtype dtype,
                             int64_t vocab, int64_t dim, const int64_t *tokens, int64_t rows,
                             int64_t ignore_index, float scale, void *out, int64_t out_row_stride,
                             int32_t *dev_status, void *stream);

gbce_status embedding_lookup_bwd(const void *grad_out, int64_t grad_row_stride, gbce_dtype dtype,
                                 int64_t rows, int64_t dim, const int64_t *tokens, int64_t vocab,
                                 int64_t ignore_index, float scale, void *dtable,
                                 int64_t dtable_row_stride, int accumulate, void *workspace,
                                 size_t workspace_bytes, int32_t *dev_status, void *stream);

/*
 * The losses of post-training, from the same [rows, vocab] logits: z = x / T,
 * q = softmax(z) over the row's vocab columns.  A row that is left out
 * (row_mask[r] == 0, or label == ignore_index) has loss 0 and a zero gradient
 * row whatever it holds; its logits are not read.  Columns masked with -inf or
 * with the type's lowest value have no mass beside others (a row that is at the
 * lowest value throughout is uniform; one that is -inf throughout, or has a NaN
 * or a +inf, has no softmax: NaN).  Sums over rows are taken
 * with 48 bits in a fixed order; row losses and gradients are fp32 throughout,
 * dlogits rounded once.  workspace: gbce_workspace_size(rows, vocab, 1) bytes
 * unless stated, 16-byte aligned, of one call at a time (a captured graph
 * keeps its own); nothing in it needs zeroing.  The temperature is a double,
 * in [1e-30, 1e30]: rounded to fp32 it would move every log p of a sequence in
 * one direction.
 *
 * Source: the calls that the pages' log-probs and cross-entropies serve are
 * the RL and preference trainers of "perf(rlhf): chunk selective_log_softmax
 * instead of looping per token", "PR information", and the distillation
 * losses of "Fix softmax collapse in CE, GRPO, KL/JSD and softmax",
 * "Summary"; the formulas are written out here.
 */

/* Largest number of teacher entries per row. */
#define GBCE_MAX_TEACHER_K 256

/*
 * Distillation from a teacher's top logits.  Row r lists the teacher's
 * columns index[r, k] (-1: no entry, its teacher logit unread) and its logits
 * t[r, k] there; teacher_rest[r], where given, is log sum_j e^{t_j / T} over
 * the teacher's other columns (-inf: none).  With p the softmax over t / T of
 * the entries and the rest,
 *   loss_r = sum_k p_k (log p_k - log q_k) + p_rest (log p_rest - log q_rest),
 *   q_rest = the sum of q over the columns not listed,
 *   dz_k = q_k - p_k (listed),   dz_j = (q_rest - p_rest) q_j / q_rest (others),
 *   dlogits = g_r dz / T,
 * 0 log 0 = 0, g_r = grad_out[r] (NONE), grad_out[0] (SUM) or grad_out[0] /
 * n_items (MEAN, n_items the rows not masked out).  Without teacher_rest the
 * teacher is its listed entries renormalised and dz = q - p.  The loss is
 * evaluated as sum p (q / p - 1 - log (q / p)), whose terms are not negative,
 * and q - p as p expm1(log q - log p): a student close to its teacher keeps
 * both.  A column listed twice counts once, with the sum of both
 * probabilities.  A row without entries, or whose entries are all -inf,
 * and without a rest has loss 0 and a zero gradient (it is still counted).  A
 * teacher logit of -inf has p = 0; a NaN or +inf one, or such a teacher_rest,
 * makes the row's loss and gradient NaN.  (The conventional factor T^2 of
 * softened teachers belongs in grad_out.)
 *
 *   index          [rows, k] int64, 1 <= k <= GBCE_MAX_TEACHER_K
 *   teacher_logits [rows, k] fp32
 *   teacher_rest   [rows] fp32 or NULL
 *   loss_out       [rows] (NONE) or [1]
 *   rest_state_out [rows, 2] fp32 or NULL: the max m over the row's unlisted
 *                  columns (raw logits) and sum e^{(x_j - m) / T}; distill_bwd
 *                  takes it back (a row left out: -inf, 0)
 *   n_items_out    [1] int64 or NULL
 * Errors: as the cross-entropy calls; an index other than -1 outside
 * [0, vocab) sets GBCE_DEV_BAD_INDEX and makes the row's loss and gradient
 * NaN.
 */
gbce_status distill_fwd(const void *logits, gbce_dtype dtype, int64_t rows, int64_t vocab,
                        int64_t row_stride, const int64_t *index, int64_t k,
                        const float *teacher_logits, const float *teacher_rest, double temperature,
                        const uint8_t *row_mask, gbce_reduction reduction, float *loss_out,
                        float *rest_state_out, int64_t *n_items_out, void *workspace,
                        size_t workspace_bytes, int32_t *dev_status, void *stream);

/* The gradient from distill_fwd's rest state (same logits, teacher and T). */
gbce_status distill_bwd(const void *logits, gbce_dtype dtype, int64_t rows, int64_t vocab,
                        int64_t row_stride, const int64_t *index, int64_t k,
                        const float *teacher_logits, const float *teacher_rest, double temperature,
                        const uint8_t *row_mask, gbce_reduction reduction, const float *grad_out,
                        const float *rest_state, const int64_t *n_items, void *dlogits,
                        int64_t dlogits_row_stride, int32_t *dev_status, void *stream);

/* Loss and gradient in one call, each row read from HBM once. */
gbce_status distill_fwd_bwd_fused(const void *logits, gbce_dtype dtype, int64_t rows,
                                  int64_t vocab, int64_t row_stride, const int64_t *index,
                                  int64_t k, const float *teacher_logits,
                                  const float *teacher_rest, double temperature,
                                  const uint8_t *row_mask, gbce_reduction reduction,
                                  const float *grad_out, float *loss_out, int64_t *n_items_out,
                                  void *dlogits, int64_t dlogits_row_stride, void *workspace,
                                  size_t workspace_bytes, int32_t *dev_status, void *stream);

/*
 * The clipped policy loss with a KL term.  With lp = log q_y of the row's
 * token, A its advantage, rho = e^{lp - old_logp} (1 without old_logp: the
 * current policy is the old one) and d = ref_logp - lp:
 *   loss_r = -min(rho A, clip(rho, 1 - clip_low, 1 + clip_high) A)
 *            + kl_beta (e^d - 1 - d),
 *   dloss_r/dlp = -rho A (0 where the clip holds) - kl_beta (e^d - 1);
 * at a clip's border itself the gradient is the unclipped one, and a row with
 * A = 0 has no surrogate, however large its ratio.
 *   clip_low in [0, 1], clip_high >= 0 (may be +inf: no clip),
 *   kl_beta >= 0; ref_logp may be NULL only when kl_beta is 0.
 */
typedef struct gbce_policy_options {
    float clip_low;
    float clip_high;
    float kl_beta;
} gbce_policy_options;

/*
 * From log-probs (of selective_logsoftmax, linear_selective_logsoftmax or
 * vocab_slice_combine with k = 1): loss, and dlogp_out[r] = the derivative by
 * logp[r] times the upstream gradient, which those calls' backward takes as
 * grad_logp.  All of logp, advantages, old_logp, ref_logp and dlogp_out are
 * [rows] fp32; rows with row_mask[r] == 0 give 0 whatever they hold.  dlogp_out
 * may be NULL (then grad_out too).  workspace: gbce_workspace_size(rows, 1, 1).
 */
gbce_status policy_loss(const float *logp, int64_t rows, const uint8_t *row_mask,
                        const float *advantages, const float *old_logp, const float *ref_logp,
                        const gbce_policy_options *options, gbce_reduction reduction,
                        const float *grad_out, float *loss_out, float *dlogp_out,
                        int64_t *n_items_out, void *workspace, size_t workspace_bytes,
                        void *stream);

/*
 * From logits, loss and dlogits in one call (each row read from HBM once):
 * lp = log q_{labels[r]}, rows with label == ignore_index left out; reductions
 * as in ce_fwd; logp_out [rows] or NULL.  Errors as ce_fwd_bwd_fused.
 */
gbce_status policy_loss_fwd_bwd_fused(const void *logits, gbce_dtype dtype, int64_t rows,
                                      int64_t vocab, int64_t row_stride, const int64_t *labels,
                                      int64_t ignore_index, double temperature,
                                      const float *advantages, const float *old_logp,
                                      const float *ref_logp, const gbce_policy_options *options,
                                      gbce_reduction reduction, const float *grad_out,
                                      float *loss_out, float *logp_out, int64_t *n_items_out,
                                      void *dlogits, int64_t dlogits_row_stride, void *workspace,
                                      size_t workspace_bytes, int32_t *dev_status, void *stream);

/*
 * The preference loss of paired sequences.  The rows are the tokens of 2 pairs
 * sequences laid end to end: sequence s has rows [seq_offsets[s],
 * seq_offsets[s + 1]), the chosen answers first (s < pairs), then the rejected
 * ones in the same order.  A sequence's score is
 *   score_s = sum over its live rows of (lp_r - ref_logp_r)
 * (ref_logp NULL: 0; `average`: divided by the number of live rows, at least
 * 1), h_i = score_i - score_{pairs + i}, and with sigma the logistic function
 *   GBCE_PREFERENCE_SIGMOID: loss_i = -(1 - eps) log sigma(u) - eps log sigma(-u),
 *                            u = beta (h_i - margin), eps = label_smoothing,
 *   GBCE_PREFERENCE_SQUARED: loss_i = (h_i - 1 / (2 beta))^2.
 * A sequence may be empty, or all of its rows left out (score 0).  Rows before
 * the first sequence or behind the last have no part in anything (log p 0, a
 * zero gradient).  Scores are summed with 48 bits.
 * Reductions are over pairs (MEAN: / pairs).  Offsets are device memory: where
 * one decreases or leaves [0, rows], sequences may overlap, and the call sets
 * GBCE_DEV_BAD_INDEX and makes every loss, every score and the gradient of every
 * live row from the first offset to the last NaN; no access leaves the rows.
 *   beta > 0; label_smoothing in [0, 0.5); margin and label_smoothing 0 with
 *   GBCE_PREFERENCE_SQUARED.
 */
typedef enum {
    GBCE_PREFERENCE_SIGMOID = 0,
    GBCE_PREFERENCE_SQUARED = 1
} gbce_preference_kind;

typedef struct gbce_preference_options {
    float beta;
    float margin;
    float label_smoothing;
    int32_t kind;
    int32_t average;
} gbce_preference_options;

/* Workspace of the two preference calls, a pure function of its arguments;
 * 0 for arguments that no call takes. */
size_t gbce_preference_workspace_size(int64_t rows, int64_t pairs);

/*
 * From log-probs, as policy_loss.  seq_offsets [2 pairs + 1] int64, grad_out
 * [pairs] (NONE) or [1], seq_score_out [2 pairs] or NULL, dlogp_out [rows] or
 * NULL (then grad_out may be NULL too).
 */
gbce_status preference_loss(const float *logp, int64_t rows, const uint8_t *row_mask,
                            const int64_t *seq_offsets, int64_t pairs, const float *ref_logp,
                            const gbce_preference_options *options, gbce_reduction reduction,
                            const float *grad_out, float *loss_out, float *dlogp_out,
                            float *seq_score_out, void *workspace, size_t workspace_bytes,
                            int32_t *dev_status, void *stream);

/*
 * From logits, loss and dlogits in one call.  A row's gradient needs its whole
 * pair's scores, so the logits are read twice.
 */
gbce_status preference_loss_fwd_bwd_fused(
    const void *logits, gbce_dtype dtype, int64_t rows, int64_t vocab, int64_t row_stride,
    const int64_t *labels, int64_t ignore_index, double temperature, const int64_t *seq_offsets,
    int64_t pairs, const float *ref_logp, const gbce_preference_options *options,
    gbce_reduction reduction, const float *grad_out, float *loss_out, float *logp_out,
    float *seq_score_out, void *dlogits, int64_t dlogits_row_stride, void *workspace,
    size_t workspace_bytes, int32_t *dev_status, void *stream);

/*
 * ce_fwd_bwd_fused without a caller workspace and without any allocation.
 *
 * The pages have no counterpart: this exists for callers that cannot provide
 * scratch memory -- a C program or plugin without a device allocator of its
 * own, which must not call cudaMalloc on its hot path (cudaMalloc can
 * synchronize the device, and next to a framework's caching allocator it can
 * fail or fragment memory).  The scratch is a fixed array of
 * GBCE_NOALLOC_SCRATCH_BYTES bytes inside the library's device image, held on
 * every GPU that loads the library until the process exits.
 *
 * Arguments and results are those of ce_fwd_bwd_fused minus the workspace.
 * Returns GBCE_EWORKSPACE, before any GPU work, when
 * gbce_workspace_size(rows, vocab, 1) > GBCE_NOALLOC_SCRATCH_BYTES (about
 * 130 000 rows).  The first call on each device looks up the array's device
 * address (cudaGetSymbolAddress) with that device current and keeps it for
 * the rest of the process; make that first call before any stream capture.
 * The kept address belongs to the device's primary context as it was then:
 * after cudaDeviceReset (or any other reset of that context) it is stale,
 * so a program that resets a device must not call this entry point on it
 * afterwards.  All calls share the one array: calls whose GPU work overlaps
 * (e.g. on two streams) race and must be serialized by the caller.  Nothing
 * in the array needs zeroing beforehand: each call writes every scratch
 * value it reads (the item count, the row ticket, the per-row losses) first.
 */
#define GBCE_NOALLOC_SCRATCH_BYTES (1u << 20)
gbce_status ce_fwd_bwd_fused_noalloc(const void *logits, gbce_dtype dtype, int64_t rows,
                                     int64_t vocab, int64_t row_stride, const int64_t *labels,
                                     int64_t ignore_index, float temperature,
                                     gbce_reduction reduction, const float *grad_out,
                                     float *loss_out, float *logp_out, float *lse_out,
                                     int64_t *n_items_out, void *dlogits,
                                     int64_t dlogits_row_stride, int32_t *dev_status,
                                     void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GBCE_H */
