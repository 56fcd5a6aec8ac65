// Internal interface between the C-ABI layer of the post-training losses
// (gbce_post_api.cu) and their row kernels (one translation unit per logit
// type).  Not installed, not part of the ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gbce {

constexpr int kMaxListed = 256;  // teacher entries of a row (GBCE_MAX_TEACHER_K)

// Which loss a row kernel computes, how much of it, and by CTAs of which shape.
enum PostOp : int {
    kOpDistill = 0,
    kOpPolicy = 1,
    kOpToken = 2,  // log p of one column and its gradient (around the preference loss)
};
enum PostPass : int { kPassFwd = 0, kPassBwd = 1, kPassFused = 2 };
enum ShapeOfCta : int { kShapeShort = 0, kShapeMid = 1, kShapeLong = 2 };

// The clipped policy loss of one row (see policy_row).
struct PolicyTerms {
    const float *advantages;  // [rows]
    const float *old_logp;    // [rows] or null (the current log p, held constant)
    const float *ref_logp;    // [rows] or null (no KL term)
    float clip_low, clip_high, kl_beta;
};

struct PostParams {
    const void *logits;
    int64_t rows, vocab, row_stride;  // row_stride in elements
    float c_hi, c_lo;                 // log2(e) / T in two floats
    float it_hi, it_lo;               // 1 / T in two floats
    float far;                        // logits from here on have |x| log2(e) / T >= 2^31

    // distillation: the teacher's entries
    const int64_t *index;       // [rows, k] columns, -1: no entry
    const float *teacher;       // [rows, k] logits
    const float *teacher_rest;  // [rows] log-sum-exp of its other logits / T, or null
    int64_t k;
    const uint8_t *row_mask;  // [rows] or null

    // policy, token
    const int64_t *labels;  // [rows]
    int64_t ignore_index;
    PolicyTerms policy;
    // token: rows outside [row_range[0], row_range[row_range_end]) are left out; null: none
    const int64_t *row_range;
    int64_t row_range_end;

    float *loss_rows;         // distill, policy: [rows] (null in the backward pass)
    float *logp_out;          // policy, token: [rows] or null
    float *rest_state_out;    // forward: [rows, 2] (m, s) of the unlisted columns, or null
    const float *rest_state;  // backward: the forward's

    void *dlogits;
    int64_t d_stride;
    const float *grad_out;  // [rows] or [1]
    int reduction;          // 0 none, 1 sum, 2 mean
    const int64_t *n_items;   // backward: the forward's count
    int64_t *n_items_out;     // else: the count goes here (null: not wanted)
    int32_t *dev_status;
    int32_t *ticket;    // hands out the rows beyond the first wave
    int32_t *zero_out;  // zeroed on the way, nullable
    int splits;       // CTAs (a cluster) per row
    int64_t keep_from;  // forward: rows from here on stay in L2 for a backward pass that follows
    int reverse;      // walk the rows from the last to the first
};

template <typename T>
cudaError_t launch_post(const PostParams &p, int op, int pass, cudaStream_t stream);

// The same for short rows (gbce_post_short.cuh).
template <typename T>
cudaError_t launch_post_short(const PostParams &p, int op, int pass, cudaStream_t stream);

// Bytes of a row up to which it goes there, unless it is one of a few and longer
// than kShortAlwaysBytes.  Two CTAs of the longest fit an SM.  Streamed / kept, us:
// policy loss, 4000 x 8192 bf16 50 / 29, 1922 x 32768 52 / 48, 8000 x 35000 198 / 182, 4000 x
// 50000 135 / 140; preference loss, 4000 x 50000 174 / 173; distillation, 8192 x 2000 114 / 24,
// 8192 x 32768 205 / 186, 1000 x 40000 47 / 41, 4000 x 40000 124 / 130; of 140 KB and more:
// policy loss, 8000 x 70000 363 / 488, 1500 x 100000 117 / 132.
constexpr int64_t kShortRowBytes = 104 * 1024, kShortAlwaysBytes = 64 * 1024, kShortFewest = 16;
// ... to one warp (where there are more rows than kShortFewRows), to four, to
// eight.  One / four / eight warps, us: policy loss, 8192 x 300 bf16 12 / 30 / 54, 8192 x
// 4000 30 / 39 / 64, 4000 x 8192 30 / 29 / 39, 8000 x 12000 80 / 68 / 87; preference loss,
// 4000 x 20000 - / 72 / 75; policy loss, 1922 x 32768 - / 50 / 48.  Few rows: distillation,
// 100 x 3000 one warp 8.0, four 6.7; 1000 x 2000 9.0, 9.5.
constexpr int64_t kShortWarpBytes = 8192, kShortMidBytes = 49152, kShortFewRows = 400;
// The most shared memory a CTA of theirs takes.
constexpr int kShortSmemMax = kShortRowBytes + 64 + 8 * kMaxListed;

// n_items = number of rows with mask != 0 (rows when mask is null) into *n_out;
// *zero_out (nullable) is zeroed.
cudaError_t launch_count_mask(const uint8_t *mask, int64_t rows, int64_t *n_out,
                              int32_t *zero_out, cudaStream_t stream);

// loss_out[0] = sum of the rows' losses, or (mean) that over *n_items, 0 for no
// items; in a fixed order.
cudaError_t launch_sum_rows(const float *loss_rows, int64_t rows, int mean, const int64_t *n_items,
                            float *loss_out, cudaStream_t stream);

}  // namespace gbce
