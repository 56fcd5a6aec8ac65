// C-ABI entry points of the post-training losses (declared in include/gbce.h):
// argument checks and dispatch, and the small kernels that work on per-row
// values only (rows counted, the policy loss of given log-probs, the
// preference loss of paired sequences).  No entry point allocates memory or
// synchronizes the host.
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gbce_post.cuh"

namespace gbce {

// -------------------------------------------------------------- rows counted

constexpr int kCountThreads = 256;

__global__ void __launch_bounds__(kCountThreads)
    count_mask_kernel(const uint8_t *mask, int64_t rows, int64_t *n_out)
{
    __shared__ int64_t part[kCountThreads / 32];
    int64_t n = 0;
    if (mask == nullptr)
        n = threadIdx.x == 0 ? rows : 0;
    else
        for (int64_t r = threadIdx.x; r < rows; r += kCountThreads)
            n += mask[r] != 0;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        n += __shfl_xor_sync(0xffffffffu, n, off);
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = n;
    __syncthreads();
    if (threadIdx.x == 0) {
        n = 0;
        for (int w = 0; w < kCountThreads / 32; ++w)
            n += part[w];
        *n_out = n;
    }
}

cudaError_t launch_count_mask(const uint8_t *mask, int64_t rows, int64_t *n_out,
                              cudaStream_t stream)
{
    count_mask_kernel<<<1, kCountThreads, 0, stream>>>(mask, rows, n_out);
    note_launches(1);
    return cudaGetLastError();
}

// ------------------------------------------- policy loss of given log-probs

// One thread per row: 17 to 21 bytes of traffic and some twenty operations.
__global__ void __launch_bounds__(256)
    policy_logp_kernel(const float *logp, int64_t rows, const uint8_t *mask, PolicyTerms t,
                       int reduction, const float *grad_out, const int64_t *n_items,
                       float *loss_rows, float *dlogp)
{
    const int64_t r = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (r >= rows)
        return;
    float loss = 0.0f, d = 0.0f;
    if (mask == nullptr || mask[r] != 0) {
        policy_row(t, r, logp[r], loss, d);
        if (dlogp != nullptr) {
            float g = reduction == 0 ? grad_out[r] : grad_out[0];
            if (reduction == 2)
                g /= static_cast<float>(*n_items);  // (this row is live: the count is not 0)
            d *= g;
        }
    }
    if (loss_rows != nullptr)
        loss_rows[r] = loss;
    if (dlogp != nullptr)
        dlogp[r] = d;
}

// -------------------------------------------------------------- preference

// A sequence's rows, [lo, hi), clamped into [0, rows]: whatever the offsets
// hold, no access leaves the rows.
struct SeqRows {
    int64_t lo, hi;
};

__device__ __forceinline__ SeqRows seq_rows(const int64_t *offsets, int64_t s, int64_t rows)
{
    const int64_t a = offsets[s], b = offsets[s + 1];
    SeqRows q;
    q.lo = a < 0 ? 0 : (a > rows ? rows : a);
    q.hi = b < 0 ? 0 : (b > rows ? rows : b);
    return q;
}

// The labels as the sweeps take them: ignore_index for rows of no sequence.
// Offsets that decrease or leave [0, rows] are reported (bad_offsets is also
// left for the pair kernel, which then makes the losses NaN).
__global__ void __launch_bounds__(256)
    preference_labels_kernel(const int64_t *labels, int64_t rows, int64_t ignore_index,
                             const int64_t *offsets, int64_t sequences, int64_t *out)
{
    const int64_t r = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (r < rows)
        out[r] = r >= offsets[0] && r < offsets[sequences] ? labels[r] : ignore_index;
}

struct PreferenceTerms {
    const float *logp;      // [rows]
    const float *ref_logp;  // [rows] or null
    int64_t rows, pairs;
    const int64_t *offsets;  // [2 pairs + 1]
    // live rows: labels[r] != ignore_index, or mask[r] != 0, or all
    const int64_t *labels;
    int64_t ignore_index;
    const uint8_t *mask;
    double beta, margin, eps;
    int squared, average;
    int reduction;
    const float *grad_out;  // [pairs] or [1]
    float sign;             // of the rows' gradients: +1 d/dlogp, -1 as token CE's upstream
    float *loss_pairs;      // [pairs]
    float *seq_score;       // [2 pairs] or null
    float *drow;            // [rows] or null
    int32_t *dev_status;
};

constexpr int kPairThreads = 256;

__device__ __forceinline__ bool preference_live(const PreferenceTerms &t, int64_t r)
{
    if (t.labels != nullptr)
        return t.labels[r] != t.ignore_index;
    return t.mask == nullptr || t.mask[r] != 0;
}

// Sum over the CTA in a fixed tree, to every thread.
__device__ double cta_sum(double v, double *scratch)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, off);
    if ((threadIdx.x & 31) == 0)
        scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
    for (int w = 0; w < kPairThreads / 32; ++w)
        v += scratch[w];
    __syncthreads();
    return v;
}

// One CTA per pair: the scores of its two sequences, summed in fp64 in a fixed
// order (a sum of thousands of log-probs meets another of the same size), the
// pair's loss, and the derivative by each of its rows' log-probs.
__global__ void __launch_bounds__(kPairThreads) preference_pair_kernel(const PreferenceTerms t)
{
    __shared__ double scratch[kPairThreads / 32];
    const int tid = threadIdx.x;
    const int64_t i = blockIdx.x;
    double score[2], weight[2];
    bool bad = t.offsets[0] < 0 || t.offsets[2 * t.pairs] > t.rows;
    SeqRows q[2];
    for (int side = 0; side < 2; ++side) {
        const int64_t s = i + side * t.pairs;
        q[side] = seq_rows(t.offsets, s, t.rows);
        bad |= t.offsets[s] > t.offsets[s + 1] || t.offsets[s] < 0 || t.offsets[s + 1] > t.rows;
        double sum = 0.0, count = 0.0;
        for (int64_t r = q[side].lo + tid; r < q[side].hi; r += kPairThreads)
            if (preference_live(t, r)) {
                const double ref = t.ref_logp != nullptr ? t.ref_logp[r] : 0.0;
                sum += static_cast<double>(t.logp[r]) - ref;
                count += 1.0;
            }
        sum = cta_sum(sum, scratch);
        count = cta_sum(count, scratch);
        weight[side] = t.average ? 1.0 / (count > 1.0 ? count : 1.0) : 1.0;
        score[side] = sum * weight[side];
    }
    // loss and dloss/dh, h the difference of the scores
    const double h = score[0] - score[1];
    double loss, dh;
    if (t.squared) {
        const double e = h - 0.5 / t.beta;
        loss = e * e;
        dh = 2.0 * e;
    } else {
        // -(1 - eps) log sig(z) - eps log sig(-z) = softplus(-z) + eps z
        const double z = t.beta * (h - t.margin), e = exp(-fabs(z));
        const double small = e / (1.0 + e);           // sig(-|z|)
        const double other = z > 0.0 ? small : 1.0 - small;  // sig(-z)
        loss = (z > 0.0 ? 0.0 : -z) + log1p(e) + (t.eps != 0.0 ? t.eps * z : 0.0);
        dh = t.beta * (t.eps - other);
    }
    if (bad) {
        loss = dh = __longlong_as_double(0x7ff8000000000000ll);
        if (tid == 0)
            report(t.dev_status, GBCE_DEV_BAD_INDEX);
    }
    if (tid == 0) {
        t.loss_pairs[i] = static_cast<float>(loss);
        if (t.seq_score != nullptr) {
            t.seq_score[i] = static_cast<float>(score[0]);
            t.seq_score[i + t.pairs] = static_cast<float>(score[1]);
        }
    }
    if (t.drow == nullptr)
        return;
    double g = t.reduction == 0 ? t.grad_out[i] : t.grad_out[0];
    if (t.reduction == 2)
        g /= static_cast<double>(t.pairs);
    for (int side = 0; side < 2; ++side) {
        const double d = (side == 0 ? dh : -dh) * weight[side] * g * t.sign;
        for (int64_t r = q[side].lo + tid; r < q[side].hi; r += kPairThreads)
            t.drow[r] = preference_live(t, r) ? static_cast<float>(d) : 0.0f;
    }
}

// loss_out[0] = sum of n losses, or their mean, in fp64 and a fixed order.
__global__ void __launch_bounds__(kPairThreads)
    pair_reduce_kernel(const float *loss, int64_t n, int mean, float *loss_out)
{
    __shared__ double scratch[kPairThreads / 32];
    double sum = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kPairThreads)
        sum += static_cast<double>(loss[i]);
    sum = cta_sum(sum, scratch);
    if (threadIdx.x == 0)
        *loss_out = static_cast<float>(mean ? sum / static_cast<double>(n) : sum);
}

// Zeros for the rows of no sequence (a preference call from log-probs).
__global__ void __launch_bounds__(256)
    preference_outside_kernel(int64_t rows, const int64_t *offsets, int64_t sequences, float *drow)
{
    const int64_t r = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (r < rows && (r < offsets[0] || r >= offsets[sequences]))
        drow[r] = 0.0f;
}

}  // namespace gbce

using gbce::PostParams;
using gbce::PreferenceTerms;

namespace {

constexpr int64_t kMaxVocab = INT32_MAX - 64;  // columns are int32 on the device
constexpr int64_t kMaxRows = INT32_MAX / 8;    // as the cross-entropy calls'

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
size_t elem_size(gbce_dtype dt) { return dt == GBCE_BF16 ? 2 : 4; }
gbce_status cuda_status(cudaError_t e) { return e == cudaSuccess ? GBCE_OK : GBCE_ECUDA; }

bool good_reduction(gbce_reduction r) { return r == GBCE_NONE || r == GBCE_SUM || r == GBCE_MEAN; }

gbce_status check_logits(const void *logits, gbce_dtype dtype, int64_t rows, int64_t vocab,
                         int64_t row_stride, float temperature)
{
    if (dtype != GBCE_F32 && dtype != GBCE_BF16)
        return GBCE_EDTYPE;
    if (rows < 0 || rows > kMaxRows || vocab < 1 || vocab > kMaxVocab || row_stride < vocab)
        return GBCE_EINVAL;
    if (!(std::isfinite(temperature) && temperature > 0.0f))
        return GBCE_EINVAL;
    if (rows == 0)
        return GBCE_OK;
    if (logits == nullptr || row_stride > (INT64_MAX / 8) / rows)
        return GBCE_EINVAL;
    if (reinterpret_cast<uintptr_t>(logits) % elem_size(dtype) != 0)
        return GBCE_EDTYPE;
    return GBCE_OK;
}

gbce_status check_dlogits(const void *logits, gbce_dtype dtype, int64_t rows, int64_t vocab,
                          int64_t row_stride, const void *dlogits, int64_t d_stride)
{
    if (dlogits == nullptr || d_stride < vocab || d_stride > (INT64_MAX / 8) / rows)
        return GBCE_EINVAL;
    const size_t es = elem_size(dtype);
    if (reinterpret_cast<uintptr_t>(dlogits) % es != 0)
        return GBCE_EDTYPE;
    const uintptr_t a = reinterpret_cast<uintptr_t>(logits);
    const uintptr_t b = reinterpret_cast<uintptr_t>(dlogits);
    const size_t na = static_cast<size_t>((rows - 1) * row_stride + vocab) * es;
    const size_t nb = static_cast<size_t>((rows - 1) * d_stride + vocab) * es;
    return a < b + nb && b < a + na ? GBCE_EINVAL : GBCE_OK;
}

gbce_status check_workspace(const void *ws, size_t bytes, size_t need)
{
    if (need == 0)
        return GBCE_OK;
    if (ws == nullptr || bytes < need || reinterpret_cast<uintptr_t>(ws) % 16 != 0)
        return GBCE_EWORKSPACE;
    return GBCE_OK;
}

PostParams post_params(const void *logits, int64_t rows, int64_t vocab, int64_t row_stride,
                       float temperature, int32_t *dev_status)
{
    PostParams p{};
    p.logits = logits;
    p.rows = rows;
    p.vocab = vocab;
    p.row_stride = row_stride;
    p.T = temperature;
    // log2(e) / T rounded once from the fp64 quotient
    p.c = static_cast<float>(1.4426950408889634 / static_cast<double>(temperature));
    p.dev_status = dev_status;
    return p;
}

void set_dlogits(PostParams &p, gbce_dtype dt, void *dlogits, int64_t d_stride)
{
    const uint64_t es = elem_size(dt);
    p.dlogits = dlogits;
    p.d_stride = d_stride;
    // every dlogits row at its logits row's offset modulo 16 bytes
    p.vec_store = ((reinterpret_cast<uintptr_t>(p.logits) ^ reinterpret_cast<uintptr_t>(dlogits)) &
                   15u) == 0 &&
                  ((static_cast<uint64_t>(p.row_stride) * es) & 15u) ==
                      ((static_cast<uint64_t>(d_stride) * es) & 15u);
}

cudaError_t launch_post(const PostParams &p, gbce_dtype dt, int op, int pass, cudaStream_t s)
{
    return dt == GBCE_BF16 ? gbce::launch_post<__nv_bfloat16>(p, op, pass, s)
                           : gbce::launch_post<float>(p, op, pass, s);
}

// Workspace of the per-row losses: the item count, then [rows] floats.
size_t loss_workspace(int64_t rows)
{
    return rows <= 0 ? 0 : 256 + align_up(static_cast<size_t>(rows) * sizeof(float), 256);
}

template <typename P>
P *ws_at(void *ws, size_t off)
{
    return reinterpret_cast<P *>(static_cast<char *>(ws) + off);
}

// A call without rows: loss 0, no items.
cudaError_t empty_loss(gbce_reduction reduction, float *loss_out, int64_t *n_items_out,
                       cudaStream_t s)
{
    if (reduction != GBCE_NONE)
        return gbce::launch_reduce_loss(nullptr, nullptr, 0, 0, static_cast<int>(reduction),
                                        nullptr, n_items_out, loss_out, s);
    return n_items_out != nullptr ? gbce::launch_count_mask(nullptr, 0, n_items_out, s)
                                  : cudaSuccess;
}

gbce_status check_policy(const gbce_policy_options *o)
{
    if (o == nullptr || !(o->clip_low >= 0.0f && o->clip_low <= 1.0f) || !(o->clip_high >= 0.0f) ||
        !(o->kl_beta >= 0.0f && std::isfinite(o->kl_beta)))
        return GBCE_EINVAL;
    return GBCE_OK;
}

gbce::PolicyTerms policy_terms(const gbce_policy_options *o, const float *advantages,
                               const float *old_logp, const float *ref_logp)
{
    return {advantages, old_logp, ref_logp, o->clip_low, o->clip_high, o->kl_beta};
}

gbce_status check_preference(const gbce_preference_options *o)
{
    if (o == nullptr || (o->kind != GBCE_PREFERENCE_SIGMOID && o->kind != GBCE_PREFERENCE_SQUARED))
        return GBCE_EINVAL;
    if (!(o->beta > 0.0f && std::isfinite(o->beta)) || !std::isfinite(o->margin))
        return GBCE_EINVAL;
    // sums of losses that each kind does not have
    if (o->kind == GBCE_PREFERENCE_SQUARED && (o->margin != 0.0f || o->label_smoothing != 0.0f))
        return GBCE_EINVAL;
    if (!(o->label_smoothing >= 0.0f && o->label_smoothing < 0.5f))
        return GBCE_EINVAL;
    return GBCE_OK;
}

void set_preference_options(PreferenceTerms &t, const gbce_preference_options *o)
{
    t.beta = o->beta;
    t.margin = o->margin;
    t.eps = o->label_smoothing;
    t.squared = o->kind == GBCE_PREFERENCE_SQUARED;
    t.average = o->average != 0;
}

struct PreferenceLayout {
    size_t labels, logp, grad, loss, total;
};

PreferenceLayout preference_layout(int64_t rows, int64_t pairs)
{
    const size_t r = static_cast<size_t>(rows), n = static_cast<size_t>(pairs);
    PreferenceLayout w{};
    w.loss = 0;  // (and more than the workspace that ce_fwd asks for in all)
    w.labels = 256 + align_up(n * sizeof(float), 256);
    w.logp = w.labels + align_up(r * sizeof(int64_t), 256);
    w.grad = w.logp + align_up(r * sizeof(float), 256);
    w.total = w.grad + align_up(r * sizeof(float), 256);
    return w;
}

cudaError_t reduce_pairs(const float *loss, int64_t n, gbce_reduction reduction, float *loss_out,
                         cudaStream_t s)
{
    gbce::pair_reduce_kernel<<<1, gbce::kPairThreads, 0, s>>>(loss, n, reduction == GBCE_MEAN,
                                                              loss_out);
    gbce::note_launches(1);
    return cudaGetLastError();
}

constexpr int64_t kMaxPairs = int64_t(1) << 30;

}  // namespace

extern "C" {

// -------------------------------------------------------------- distillation

gbce_status distill_fwd(const void *logits, gbce_dtype dtype, int64_t rows, int64_t vocab,
                        int64_t row_stride, const int64_t *index, int64_t k,
                        const float *teacher_logits, const float *teacher_rest, float temperature,
                        const uint8_t *row_mask, gbce_reduction reduction, float *loss_out,
                        float *rest_state_out, int64_t *n_items_out, void *workspace,
                        size_t workspace_bytes, int32_t *dev_status, void *stream)
{
    gbce_status st = check_logits(logits, dtype, rows, vocab, row_stride, temperature);
    if (st != GBCE_OK)
        return st;
    if (k < 1 || k > GBCE_MAX_TEACHER_K || !good_reduction(reduction))
        return GBCE_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0) {
        if (reduction != GBCE_NONE && loss_out == nullptr)
            return GBCE_EINVAL;
        return cuda_status(empty_loss(reduction, loss_out, n_items_out, s));
    }
    if (index == nullptr || teacher_logits == nullptr || loss_out == nullptr)
        return GBCE_EINVAL;
    if ((st = check_workspace(workspace, workspace_bytes, loss_workspace(rows))) != GBCE_OK)
        return st;
    int64_t *n_ptr = n_items_out != nullptr ? n_items_out : ws_at<int64_t>(workspace, 0);
    PostParams p = post_params(logits, rows, vocab, row_stride, temperature, dev_status);
    p.index = index;
    p.k = k;
    p.teacher = teacher_logits;
    p.teacher_rest = teacher_rest;
    p.row_mask = row_mask;
    p.loss_rows = reduction == GBCE_NONE ? loss_out : ws_at<float>(workspace, 256);
    p.rest_state_out = rest_state_out;
    cudaError_t e = cudaSuccess;
    if (reduction == GBCE_MEAN || n_items_out != nullptr)
        e = gbce::launch_count_mask(row_mask, rows, n_ptr, s);
    if (e == cudaSuccess)
        e = launch_post(p, dtype, gbce::kOpDistill, gbce::kPassFwd, s);
    if (e == cudaSuccess && reduction != GBCE_NONE)
        e = gbce::launch_reduce_loss(p.loss_rows, nullptr, rows, 0, static_cast<int>(reduction),
                                     n_ptr, nullptr, loss_out, s);
    return cuda_status(e);
}

gbce_status distill_bwd(const void *logits, gbce_dtype dtype, int64_t rows, int64_t vocab,
                        int64_t row_stride, const int64_t *index, int64_t k,
                        const float *teacher_logits, const float *teacher_rest, float temperature,
                        const uint8_t *row_mask, gbce_reduction reduction, const float *grad_out,
                        const float *rest_state, const int64_t *n_items, void *dlogits,
                        int64_t dlogits_row_stride, int32_t *dev_status, void *stream)
{
    gbce_status st = check_logits(logits, dtype, rows, vocab, row_stride, temperature);
    if (st != GBCE_OK)
        return st;
    if (k < 1 || k > GBCE_MAX_TEACHER_K || !good_reduction(reduction))
        return GBCE_EINVAL;
    if (rows == 0)
        return GBCE_OK;
    if (index == nullptr || teacher_logits == nullptr || grad_out == nullptr ||
        rest_state == nullptr || (reduction == GBCE_MEAN && n_items == nullptr))
        return GBCE_EINVAL;
    if ((st = check_dlogits(logits, dtype, rows, vocab, row_stride, dlogits,
                            dlogits_row_stride)) != GBCE_OK)
        return st;
    PostParams p = post_params(logits, rows, vocab, row_stride, temperature, dev_status);
    p.index = index;
    p.k = k;
    p.teacher = teacher_logits;
    p.teacher_rest = teacher_rest;
    p.row_mask = row_mask;
    p.rest_state = rest_state;
    p.grad_out = grad_out;
    p.reduction = static_cast<int>(reduction);
    p.n_items = n_items;
    set_dlogits(p, dtype, dlogits, dlogits_row_stride);
    return cuda_status(launch_post(p, dtype, gbce::kOpDistill, gbce::kPassBwd,
                                   static_cast<cudaStream_t>(stream)));
}

gbce_status distill_fwd_bwd_fused(const void *logits, gbce_dtype dtype, int64_t rows,
                                  int64_t vocab, int64_t row_stride, const int64_t *index,
                                  int64_t k, const float *teacher_logits,
                                  const float *teacher_rest, float temperature,
                                  const uint8_t *row_mask, gbce_reduction reduction,
                                  const float *grad_out, float *loss_out, int64_t *n_items_out,
                                  void *dlogits, int64_t dlogits_row_stride, void *workspace,
                                  size_t workspace_bytes, int32_t *dev_status, void *stream)
{
    gbce_status st = check_logits(logits, dtype, rows, vocab, row_stride, temperature);
    if (st != GBCE_OK)
        return st;
    if (k < 1 || k > GBCE_MAX_TEACHER_K || !good_reduction(reduction))
        return GBCE_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0) {
        if (reduction != GBCE_NONE && loss_out == nullptr)
            return GBCE_EINVAL;
        return cuda_status(empty_loss(reduction, loss_out, n_items_out, s));
    }
    if (index == nullptr || teacher_logits == nullptr || grad_out == nullptr ||
        loss_out == nullptr)
        return GBCE_EINVAL;
    if ((st = check_dlogits(logits, dtype, rows, vocab, row_stride, dlogits,
                            dlogits_row_stride)) != GBCE_OK)
        return st;
    if ((st = check_workspace(workspace, workspace_bytes, loss_workspace(rows))) != GBCE_OK)
        return st;
    int64_t *n_ptr = n_items_out != nullptr ? n_items_out : ws_at<int64_t>(workspace, 0);
    PostParams p = post_params(logits, rows, vocab, row_stride, temperature, dev_status);
    p.index = index;
    p.k = k;
    p.teacher = teacher_logits;
    p.teacher_rest = teacher_rest;
    p.row_mask = row_mask;
    p.loss_rows = reduction == GBCE_NONE ? loss_out : ws_at<float>(workspace, 256);
    p.grad_out = grad_out;
    p.reduction = static_cast<int>(reduction);
    p.n_items = n_ptr;
    set_dlogits(p, dtype, dlogits, dlogits_row_stride);
    cudaError_t e = cudaSuccess;
    if (reduction == GBCE_MEAN || n_items_out != nullptr)
        e = gbce::launch_count_mask(row_mask, rows, n_ptr, s);
    if (e == cudaSuccess)
        e = launch_post(p, dtype, gbce::kOpDistill, gbce::kPassFused, s);
    if (e == cudaSuccess && reduction != GBCE_NONE)
        e = gbce::launch_reduce_loss(p.loss_rows, nullptr, rows, 0, static_cast<int>(reduction),
                                     n_ptr, nullptr, loss_out, s);
    return cuda_status(e);
}

// --------------------------------------------------------------- policy loss

gbce_status policy_loss(const float *logp, int64_t rows, const uint8_t *row_mask,
                        const float *advantages, const float *old_logp, const float *ref_logp,
                        const gbce_policy_options *options, gbce_reduction reduction,
                        const float *grad_out, float *loss_out, float *dlogp_out,
                        int64_t *n_items_out, void *workspace, size_t workspace_bytes,
                        void *stream)
{
    gbce_status st = check_policy(options);
    if (st != GBCE_OK)
        return st;
    if (rows < 0 || rows > kMaxRows || !good_reduction(reduction))
        return GBCE_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0) {
        if (reduction != GBCE_NONE && loss_out == nullptr)
            return GBCE_EINVAL;
        return cuda_status(empty_loss(reduction, loss_out, n_items_out, s));
    }
    if (logp == nullptr || advantages == nullptr || loss_out == nullptr ||
        (dlogp_out != nullptr && grad_out == nullptr) ||
        (options->kl_beta != 0.0f && ref_logp == nullptr))
        return GBCE_EINVAL;
    if ((st = check_workspace(workspace, workspace_bytes, loss_workspace(rows))) != GBCE_OK)
        return st;
    int64_t *n_ptr = n_items_out != nullptr ? n_items_out : ws_at<int64_t>(workspace, 0);
    float *loss_rows = reduction == GBCE_NONE ? loss_out : ws_at<float>(workspace, 256);
    cudaError_t e = cudaSuccess;
    if (reduction == GBCE_MEAN || n_items_out != nullptr)
        e = gbce::launch_count_mask(row_mask, rows, n_ptr, s);
    if (e == cudaSuccess) {
        gbce::policy_logp_kernel<<<static_cast<unsigned>((rows + 255) / 256), 256, 0, s>>>(
            logp, rows, row_mask, policy_terms(options, advantages, old_logp, ref_logp),
            static_cast<int>(reduction), grad_out, n_ptr, loss_rows, dlogp_out);
        gbce::note_launches(1);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess && reduction != GBCE_NONE)
        e = gbce::launch_reduce_loss(loss_rows, nullptr, rows, 0, static_cast<int>(reduction),
                                     n_ptr, nullptr, loss_out, s);
    return cuda_status(e);
}

gbce_status policy_loss_fwd_bwd_fused(const void *logits, gbce_dtype dtype, int64_t rows,
                                      int64_t vocab, int64_t row_stride, const int64_t *labels,
                                      int64_t ignore_index, float temperature,
                                      const float *advantages, const float *old_logp,
                                      const float *ref_logp, const gbce_policy_options *options,
                                      gbce_reduction reduction, const float *grad_out,
                                      float *loss_out, float *logp_out, int64_t *n_items_out,
                                      void *dlogits, int64_t dlogits_row_stride, void *workspace,
                                      size_t workspace_bytes, int32_t *dev_status, void *stream)
{
    gbce_status st = check_policy(options);
    if (st != GBCE_OK)
        return st;
    if ((st = check_logits(logits, dtype, rows, vocab, row_stride, temperature)) != GBCE_OK)
        return st;
    if (!good_reduction(reduction))
        return GBCE_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0) {
        if (reduction != GBCE_NONE && loss_out == nullptr)
            return GBCE_EINVAL;
        return cuda_status(empty_loss(reduction, loss_out, n_items_out, s));
    }
    if (labels == nullptr || advantages == nullptr || grad_out == nullptr || loss_out == nullptr ||
        (options->kl_beta != 0.0f && ref_logp == nullptr))
        return GBCE_EINVAL;
    if ((st = check_dlogits(logits, dtype, rows, vocab, row_stride, dlogits,
                            dlogits_row_stride)) != GBCE_OK)
        return st;
    if ((st = check_workspace(workspace, workspace_bytes, loss_workspace(rows))) != GBCE_OK)
        return st;
    int64_t *n_ptr = n_items_out != nullptr ? n_items_out : ws_at<int64_t>(workspace, 0);
    PostParams p = post_params(logits, rows, vocab, row_stride, temperature, dev_status);
    p.labels = labels;
    p.ignore_index = ignore_index;
    p.policy = policy_terms(options, advantages, old_logp, ref_logp);
    p.loss_rows = reduction == GBCE_NONE ? loss_out : ws_at<float>(workspace, 256);
    p.logp_out = logp_out;
    p.grad_out = grad_out;
    p.reduction = static_cast<int>(reduction);
    p.n_items = n_ptr;
    set_dlogits(p, dtype, dlogits, dlogits_row_stride);
    cudaError_t e = cudaSuccess;
    if (reduction == GBCE_MEAN || n_items_out != nullptr)
        e = gbce::launch_count_items(labels, rows, ignore_index, n_ptr, nullptr, nullptr, nullptr,
                                     s);
    if (e == cudaSuccess)
        e = launch_post(p, dtype, gbce::kOpPolicy, gbce::kPassFused, s);
    if (e == cudaSuccess && reduction != GBCE_NONE)
        e = gbce::launch_reduce_loss(p.loss_rows, nullptr, rows, 0, static_cast<int>(reduction),
                                     n_ptr, nullptr, loss_out, s);
    return cuda_status(e);
}

// ----------------------------------------------------------- preference loss

size_t gbce_preference_workspace_size(int64_t rows, int64_t pairs)
{
    if (rows < 0 || rows > kMaxRows || pairs < 1 || pairs > kMaxPairs)
        return 0;
    return preference_layout(rows, pairs).total;
}

gbce_status preference_loss(const float *logp, int64_t rows, const uint8_t *row_mask,
                            const int64_t *seq_offsets, int64_t pairs, const float *ref_logp,
                            const gbce_preference_options *options, gbce_reduction reduction,
                            const float *grad_out, float *loss_out, float *dlogp_out,
                            float *seq_score_out, void *workspace, size_t workspace_bytes,
                            int32_t *dev_status, void *stream)
{
    gbce_status st = check_preference(options);
    if (st != GBCE_OK)
        return st;
    if (rows < 0 || rows > kMaxRows || pairs < 1 || pairs > kMaxPairs ||
        !good_reduction(reduction))
        return GBCE_EINVAL;
    if (seq_offsets == nullptr || loss_out == nullptr || (rows > 0 && logp == nullptr) ||
        (dlogp_out != nullptr && grad_out == nullptr))
        return GBCE_EINVAL;
    if ((st = check_workspace(workspace, workspace_bytes,
                              preference_layout(rows, pairs).total)) != GBCE_OK)
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    PreferenceTerms t{};
    t.logp = logp;
    t.ref_logp = ref_logp;
    t.rows = rows;
    t.pairs = pairs;
    t.offsets = seq_offsets;
    t.mask = row_mask;
    set_preference_options(t, options);
    t.reduction = static_cast<int>(reduction);
    t.grad_out = grad_out;
    t.sign = 1.0f;
    t.loss_pairs = reduction == GBCE_NONE ? loss_out : ws_at<float>(workspace, 0);
    t.seq_score = seq_score_out;
    t.drow = dlogp_out;
    t.dev_status = dev_status;
    cudaError_t e = cudaSuccess;
    if (dlogp_out != nullptr && rows > 0) {
        gbce::preference_outside_kernel<<<static_cast<unsigned>((rows + 255) / 256), 256, 0, s>>>(
            rows, seq_offsets, 2 * pairs, dlogp_out);
        gbce::note_launches(1);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess) {
        gbce::preference_pair_kernel<<<static_cast<unsigned>(pairs), gbce::kPairThreads, 0, s>>>(
            t);
        gbce::note_launches(1);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess && reduction != GBCE_NONE)
        e = reduce_pairs(t.loss_pairs, pairs, reduction, loss_out, s);
    return cuda_status(e);
}

gbce_status preference_loss_fwd_bwd_fused(
    const void *logits, gbce_dtype dtype, int64_t rows, int64_t vocab, int64_t row_stride,
    const int64_t *labels, int64_t ignore_index, float temperature, const int64_t *seq_offsets,
    int64_t pairs, const float *ref_logp, const gbce_preference_options *options,
    gbce_reduction reduction, const float *grad_out, float *loss_out, float *logp_out,
    float *seq_score_out, void *dlogits, int64_t dlogits_row_stride, void *workspace,
    size_t workspace_bytes, int32_t *dev_status, void *stream)
{
    gbce_status st = check_preference(options);
    if (st != GBCE_OK)
        return st;
    if ((st = check_logits(logits, dtype, rows, vocab, row_stride, temperature)) != GBCE_OK)
        return st;
    if (pairs < 1 || pairs > kMaxPairs || !good_reduction(reduction))
        return GBCE_EINVAL;
    if (seq_offsets == nullptr || loss_out == nullptr || grad_out == nullptr ||
        (rows > 0 && labels == nullptr))
        return GBCE_EINVAL;
    if (rows > 0 && (st = check_dlogits(logits, dtype, rows, vocab, row_stride, dlogits,
                                        dlogits_row_stride)) != GBCE_OK)
        return st;
    const PreferenceLayout w = preference_layout(rows, pairs);
    if ((st = check_workspace(workspace, workspace_bytes, w.total)) != GBCE_OK)
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int64_t *kept = ws_at<int64_t>(workspace, w.labels);
    float *logp = logp_out != nullptr ? logp_out : ws_at<float>(workspace, w.logp);
    float *grad = ws_at<float>(workspace, w.grad);
    cudaError_t e = cudaSuccess;
    if (rows > 0) {
        gbce::preference_labels_kernel<<<static_cast<unsigned>((rows + 255) / 256), 256, 0, s>>>(
            labels, rows, ignore_index, seq_offsets, 2 * pairs, kept);
        gbce::note_launches(1);
        if ((e = cudaGetLastError()) != cudaSuccess)
            return GBCE_ECUDA;
        // log p of every kept row (its token CE loss goes to the gradient's place)
        st = ce_fwd(logits, dtype, rows, vocab, row_stride, kept, ignore_index, temperature,
                    GBCE_NONE, nullptr, grad, logp, nullptr, nullptr, workspace, workspace_bytes,
                    dev_status, stream);
        if (st != GBCE_OK)
            return st;
    }
    PreferenceTerms t{};
    t.logp = logp;
    t.ref_logp = ref_logp;
    t.rows = rows;
    t.pairs = pairs;
    t.offsets = seq_offsets;
    t.labels = kept;
    t.ignore_index = ignore_index;
    set_preference_options(t, options);
    t.reduction = static_cast<int>(reduction);
    t.grad_out = grad_out;
    t.sign = -1.0f;
    t.loss_pairs = reduction == GBCE_NONE ? loss_out : ws_at<float>(workspace, w.loss);
    t.seq_score = seq_score_out;
    t.drow = grad;
    t.dev_status = dev_status;
    if (e == cudaSuccess) {
        gbce::preference_pair_kernel<<<static_cast<unsigned>(pairs), gbce::kPairThreads, 0, s>>>(
            t);
        gbce::note_launches(1);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess && reduction != GBCE_NONE)
        e = reduce_pairs(t.loss_pairs, pairs, reduction, loss_out, s);
    if (e == cudaSuccess && rows > 0)
        return ce_bwd(logits, dtype, rows, vocab, row_stride, kept, ignore_index, temperature,
                      GBCE_NONE, nullptr, grad, logp, nullptr, dlogits, dlogits_row_stride,
                      dev_status, stream);
    return cuda_status(e);
}

}  // extern "C"
