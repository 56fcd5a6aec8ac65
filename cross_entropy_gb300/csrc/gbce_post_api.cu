// C-ABI entry points of the post-training losses (declared in include/gbce.h):
// argument checks and dispatch, and the small kernels that work on per-row
// values only (rows counted, the policy loss of given log-probs, the
// preference loss of paired sequences).  No entry point allocates memory or
// synchronizes the host.
#include <cfloat>
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gbce_post.cuh"

namespace gbce {

// -------------------------------------------------------------- rows counted

constexpr int kCountThreads = 256;

__global__ void __launch_bounds__(kCountThreads)
    count_mask_kernel(const uint8_t *mask, int64_t rows, int64_t *n_out, int32_t *zero_out)
{
    __shared__ int64_t part[kCountThreads / 32];
    // the row kernel after this one may start its prologue now: it waits for
    // this kernel's outputs before it reads them
    launch_dependents();
    if (threadIdx.x == 0 && zero_out != nullptr)
        *zero_out = 0;
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
                              int32_t *zero_out, cudaStream_t stream)
{
    count_mask_kernel<<<1, kCountThreads, 0, stream>>>(mask, rows, n_out, zero_out);
    note_launches(1);
    return cudaGetLastError();
}

// ---------------------------------------------------------------- losses summed

constexpr int kSumThreads = 1024, kSumWarps = kSumThreads / 32;

// Sum and count over the CTA in a fixed order, in thread 0.
__device__ __forceinline__ void cta_sum(Sum2 &s, int64_t &n, Sum2 *scratch, int64_t *counts)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int warps = blockDim.x >> 5;
    s.warp_merge();
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        n += __shfl_down_sync(0xffffffffu, n, off);
    if (lane == 0) {
        scratch[warp] = s;
        counts[warp] = n;
    }
    __syncthreads();
    if (warp == 0) {
        s = lane < warps ? scratch[lane] : Sum2{};
        n = lane < warps ? counts[lane] : 0;
        s.warp_merge();
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            n += __shfl_down_sync(0xffffffffu, n, off);
    }
}

__device__ __forceinline__ float reduced(Sum2 s, bool mean, int64_t n)
{
    const double v = s.value();
    return static_cast<float>(mean ? (n > 0 ? v / static_cast<double>(n) : 0.0) : v);
}

__global__ void __launch_bounds__(kSumThreads)
    sum_rows_kernel(const float *loss_rows, int64_t rows, int mean, const int64_t *n_items,
                    float *loss_out)
{
    __shared__ Sum2 scratch[kSumWarps];
    __shared__ int64_t counts[kSumWarps];
    // launched as a dependent of the kernel that wrote the row losses
    grid_dependency_wait();
    const int64_t kept = mean ? *n_items : 0;
    Sum2 s;
    int64_t n = 0;
#pragma unroll 8
    for (int64_t r = threadIdx.x; r < rows; r += kSumThreads)
        s.add(loss_rows[r]);
    cta_sum(s, n, scratch, counts);
    if (threadIdx.x == 0)
        *loss_out = reduced(s, mean != 0, kept);
}

cudaError_t launch_sum_rows(const float *loss_rows, int64_t rows, int mean, const int64_t *n_items,
                            float *loss_out, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kSumThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t err =
        cudaLaunchKernelEx(&cfg, sum_rows_kernel, loss_rows, rows, mean, n_items, loss_out);
    note_launches(1);
    return err != cudaSuccess ? err : cudaGetLastError();
}

// ------------------------------------------- policy loss of given log-probs

struct PolicyRows {
    const float *logp;  // [rows]
    int64_t rows;
    const uint8_t *mask;
    PolicyTerms terms;
    int reduction;
    const float *grad_out;  // [rows] or [1] or null
    float *loss_rows;       // NONE: [rows]
    float *loss_out;        // else: [1]
    float *dlogp;           // [rows] or null
    int64_t *n_items;
};

constexpr int kPolicyCtas = 8;  // of the cluster

struct ClusterSum {
    Sum2 scratch[kSumWarps];
    int64_t counts[kSumWarps];
    Sum2 cta;
    int64_t cta_count;
};

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}

// Sum and count over the cluster in a fixed order, to every thread: over each
// CTA, then the CTAs' parts in rank order.
__device__ void cluster_sum(ClusterSum &own, Sum2 &s, int64_t &n)
{
    cta_sum(s, n, own.scratch, own.counts);
    if (threadIdx.x == 0) {
        own.cta = s;
        own.cta_count = n;
    }
    cluster_barrier();
    const uint32_t a = smem_addr(&own.cta), b = smem_addr(&own.cta_count);
    s = Sum2{};
    n = 0;
#pragma unroll
    for (uint32_t i = 0; i < kPolicyCtas; ++i) {
        Sum2 v;
        int64_t k;
        asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                     : "=f"(v.hi), "=f"(v.lo)
                     : "r"(map_to_rank(a, i)));
        asm volatile("ld.shared::cluster.s64 %0, [%1];" : "=l"(k) : "r"(map_to_rank(b, i)));
        s.add(v);
        n += k;
    }
    cluster_barrier();  // (no CTA leaves, or writes its sums anew, before all have read them)
}

// Inputs of a row, read before the count is known.
struct PolicyInputs {
    float lp, adv, old_lp, ref_lp;
    bool live;
};

__device__ __forceinline__ PolicyInputs policy_inputs(const PolicyRows &q, int64_t r)
{
    PolicyInputs x = {0.0f, 0.0f, 0.0f, 0.0f, false};
    if (r < q.rows) {
        x.live = q.mask == nullptr || q.mask[r] != 0;
        x.lp = q.logp[r];
        x.adv = q.terms.advantages[r];
        x.old_lp = q.terms.old_logp != nullptr ? q.terms.old_logp[r] : 0.0f;
        x.ref_lp = q.terms.ref_logp != nullptr ? q.terms.ref_logp[r] : 0.0f;
    }
    return x;
}

// A row's loss (0 where it is left out), and its derivative stored.
__device__ __forceinline__ float policy_one_row(const PolicyRows &q, int64_t r,
                                                const PolicyInputs &x, float g)
{
    float loss = 0.0f, d = 0.0f;
    if (r >= q.rows)
        return 0.0f;
    if (x.live) {
        policy_row(q.terms, x.adv, x.old_lp, x.ref_lp, x.lp, loss, d);
        if (q.reduction == GBCE_NONE && q.dlogp != nullptr)
            g = q.grad_out[r];
        d *= g;
    }
    if (q.dlogp != nullptr)
        q.dlogp[r] = d;
    if (q.reduction == GBCE_NONE)
        q.loss_rows[r] = loss;
    return loss;
}

__device__ __forceinline__ float policy_upstream(const PolicyRows &q, int64_t n)
{
    if (q.dlogp == nullptr || q.reduction == GBCE_NONE)
        return 1.0f;
    return q.reduction == GBCE_MEAN && n > 0 ? q.grad_out[0] / static_cast<float>(n)
                                             : q.grad_out[0];
}

// One cluster for all rows: the count, the rows, the reduced loss, in one
// launch.  Latency is what such a call costs (17 to 21 bytes and some twenty
// operations a row), so the first rows' inputs are read along with the mask:
// 65536 rows took 48 us as three launches with one CTA for each of the sums.
__global__ void __cluster_dims__(kPolicyCtas, 1, 1) __launch_bounds__(kSumThreads)
    policy_cluster_kernel(const PolicyRows q)
{
    __shared__ ClusterSum sums;
    constexpr int kAhead = 4;
    constexpr int64_t kStep = static_cast<int64_t>(kPolicyCtas) * kSumThreads;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kSumThreads + threadIdx.x;
    PolicyInputs x[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        x[i] = policy_inputs(q, first + i * kStep);
    Sum2 s;
    int64_t n = 0;
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        n += x[i].live;
#pragma unroll 4
    for (int64_t r = first + kAhead * kStep; r < q.rows; r += kStep)
        n += q.mask == nullptr || q.mask[r] != 0;
    cluster_sum(sums, s, n);
    const float g = policy_upstream(q, n);
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        s.add(policy_one_row(q, first + i * kStep, x[i], g));
#pragma unroll 2
    for (int64_t r = first + kAhead * kStep; r < q.rows; r += kStep)
        s.add(policy_one_row(q, r, policy_inputs(q, r), g));
    if (first == 0)
        *q.n_items = n;
    if (q.reduction == GBCE_NONE)
        return;
    const int64_t kept = n;
    cluster_sum(sums, s, n);
    if (first == 0)
        *q.loss_out = reduced(s, q.reduction == GBCE_MEAN, kept);
}

// Many rows: a grid counts the rows of each CTA's part, a grid takes them (every
// CTA summing the parts' counts itself), one CTA sums the parts' losses.
constexpr int kPolicyPartRows = 4096, kPolicyMaxParts = 65536;

__global__ void __launch_bounds__(kSumThreads)
    policy_count_kernel(const uint8_t *mask, int64_t rows, int64_t part, int64_t *counts)
{
    __shared__ ClusterSum sums;
    const int64_t lo = blockIdx.x * part, hi = lo + part < rows ? lo + part : rows;
    Sum2 s;
    int64_t n = 0;
    for (int64_t r = lo + threadIdx.x; r < hi; r += kSumThreads)
        n += mask == nullptr || mask[r] != 0;
    cta_sum(s, n, sums.scratch, sums.counts);
    if (threadIdx.x == 0)
        counts[blockIdx.x] = n;
}

__global__ void __launch_bounds__(kSumThreads)
    policy_part_kernel(const PolicyRows q, int64_t part, const int64_t *counts, Sum2 *losses)
{
    __shared__ ClusterSum sums;
    Sum2 s;
    int64_t n = 0;
    for (int64_t i = threadIdx.x; i < gridDim.x; i += kSumThreads)
        n += counts[i];
    cta_sum(s, n, sums.scratch, sums.counts);
    if (threadIdx.x == 0)
        sums.cta_count = n;
    __syncthreads();
    n = sums.cta_count;
    const float g = policy_upstream(q, n);
    const int64_t lo = blockIdx.x * part, hi = lo + part < q.rows ? lo + part : q.rows;
    s = Sum2{};
    for (int64_t r = lo + threadIdx.x; r < hi; r += kSumThreads)
        s.add(policy_one_row(q, r, policy_inputs(q, r), g));
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *q.n_items = n;
    cta_sum(s, n, sums.scratch, sums.counts);
    if (threadIdx.x == 0)
        losses[blockIdx.x] = s;
}

__global__ void __launch_bounds__(kSumThreads)
    policy_sum_kernel(const Sum2 *losses, int64_t parts, int mean, const int64_t *n_items,
                      float *loss_out)
{
    __shared__ ClusterSum sums;
    Sum2 s;
    int64_t n = 0;
    for (int64_t i = threadIdx.x; i < parts; i += kSumThreads)
        s.add(losses[i]);
    cta_sum(s, n, sums.scratch, sums.counts);
    if (threadIdx.x == 0)
        *loss_out = reduced(s, mean != 0, *n_items);
}

// Up to this many rows go to the one cluster.
constexpr int64_t kPolicyClusterRows = 131072;

cudaError_t launch_policy_rows(const PolicyRows &q, void *parts, cudaStream_t stream)
{
    if (q.rows <= kPolicyClusterRows) {
        policy_cluster_kernel<<<kPolicyCtas, kSumThreads, 0, stream>>>(q);
        note_launches(1);
        return cudaGetLastError();
    }
    int64_t part = kPolicyPartRows;
    if ((q.rows + part - 1) / part > kPolicyMaxParts)
        part = (q.rows + kPolicyMaxParts - 1) / kPolicyMaxParts;
    const int64_t n = (q.rows + part - 1) / part;
    Sum2 *losses = static_cast<Sum2 *>(parts);
    int64_t *counts = reinterpret_cast<int64_t *>(losses + n);
    policy_count_kernel<<<static_cast<unsigned>(n), kSumThreads, 0, stream>>>(q.mask, q.rows,
                                                                                 part, counts);
    policy_part_kernel<<<static_cast<unsigned>(n), kSumThreads, 0, stream>>>(q, part, counts,
                                                                                losses);
    note_launches(2);
    if (q.reduction != GBCE_NONE) {
        policy_sum_kernel<<<1, kSumThreads, 0, stream>>>(losses, n, q.reduction == GBCE_MEAN,
                                                            q.n_items, q.loss_out);
        note_launches(1);
    }
    return cudaGetLastError();
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

struct PreferenceTerms {
    const float *logp;      // [rows]
    const float *ref_logp;  // [rows] or null
    int64_t rows, pairs;
    const int64_t *offsets;  // [2 pairs + 1]
    // live rows: labels[r] != ignore_index, or mask[r] != 0, or all
    const int64_t *labels;
    int64_t ignore_index;
    const uint8_t *mask;
    double beta, margin, half_over_beta;  // the last: 1 / (2 beta)
    float eps;
    int squared, average;
    int reduction;
    const float *grad_out;  // [pairs] or [1]
    float *loss_pairs;      // [pairs]
    float *seq_score;       // [2 pairs] or null
    float *drow;            // [rows] or null
    float *loss_out;        // reduced loss, by the last pair's CTA (null: not reduced)
    int32_t *done;          // pairs done so far, and kBadOffsets: 0 at the start
    int32_t *dev_status;
};

constexpr int kPairThreads = 256;
constexpr int32_t kBadOffsets = INT32_MIN;  // (a bit beside the count, which is at most kMaxPairs)

__device__ __forceinline__ bool preference_live(const PreferenceTerms &t, int64_t r)
{
    if (t.labels != nullptr)
        return t.labels[r] != t.ignore_index;
    return t.mask == nullptr || t.mask[r] != 0;
}

// One CTA per pair, half of it per sequence: the scores, summed in two floats in
// a fixed order (a sum of thousands of log-probs meets another of the same
// size), the pair's loss, and the derivative by each of its rows' log-probs; the
// last CTA to finish sums the losses.  All of it is latency, so the halves work
// side by side and no thread divides in FP64 unless `average` asks for it (with
// FP64 sums and functions in every thread: 18 us at two pairs of 16 rows).
__global__ void __launch_bounds__(kPairThreads) preference_pair_kernel(const PreferenceTerms t)
{
    constexpr int kWarps = kPairThreads / 32, kHalf = kPairThreads / 2;
    __shared__ Sum2 scratch[kWarps];
    __shared__ int64_t counts[kWarps];
    __shared__ float s_d[2];
    __shared__ int s_last, s_bad;
    // a dependent of the kernel that wrote the log-probs; the gradient's kernel may
    // take its place meanwhile
    launch_dependents();
    grid_dependency_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int side = tid / kHalf, first = tid - side * kHalf;
    const int64_t i = blockIdx.x, at = i + side * t.pairs;
    const SeqRows q = seq_rows(t.offsets, at, t.rows);
    bool bad = t.offsets[0] < 0 || t.offsets[2 * t.pairs] > t.rows;
    bad |= t.offsets[at] > t.offsets[at + 1] || t.offsets[at] < 0 || t.offsets[at + 1] > t.rows;
    Sum2 s;
    int64_t n = 0;
#pragma unroll 4
    for (int64_t r = q.lo + first; r < q.hi; r += kHalf)
        if (preference_live(t, r)) {
            s.add_difference(t.logp[r], t.ref_logp != nullptr ? t.ref_logp[r] : 0.0f);
            ++n;
        }
    s.warp_merge();
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        n += __shfl_down_sync(0xffffffffu, n, off);
    if (lane == 0) {
        scratch[warp] = s;
        counts[warp] = n;
    }
    bad = __syncthreads_or(bad);
    if (tid == 0) {
        double score[2];
        float weight[2];
        for (int k = 0; k < 2; ++k) {
            s = scratch[k * kWarps / 2];
            n = counts[k * kWarps / 2];
            for (int w = 1; w < kWarps / 2; ++w) {
                s.add(scratch[k * kWarps / 2 + w]);
                n += counts[k * kWarps / 2 + w];
            }
            score[k] = s.value();
            weight[k] = 1.0f;
            if (t.average && n > 1) {
                const double inv = 1.0 / static_cast<double>(n);
                score[k] *= inv;
                weight[k] = static_cast<float>(inv);
            }
        }
        // loss and dloss/dh, h the difference of the scores
        const double h = score[0] - score[1];
        float loss, dh;
        if (t.squared) {
            const float e = static_cast<float>(h - t.half_over_beta);
            loss = e * e;
            dh = 2.0f * e;
        } else {
            // -(1 - eps) log sig(z) - eps log sig(-z) = log(1 + e^-|z|) + eps z for z > 0,
            // + (1 - eps)(-z) for z < 0 (one product: z may be infinite)
            const float z = static_cast<float>(t.beta * (h - t.margin));
            const float e = expf(-fabsf(z)), small = e / (1.0f + e);  // sig(-|z|)
            loss = log1pf(e) + (z <= 0.0f ? -(1.0f - t.eps) * z : t.eps != 0.0f ? t.eps * z : 0.0f);
            // sig(-z) - eps, which for z < 0 is 1 - eps - sig(z)
            dh = static_cast<float>(-t.beta) *
                 (z > 0.0f ? small - t.eps : (1.0f - t.eps) - small);
        }
        if (bad)
            report(t.dev_status, GBCE_DEV_BAD_INDEX);
        t.loss_pairs[i] = loss;
        if (t.seq_score != nullptr) {
            t.seq_score[i] = static_cast<float>(score[0]);
            t.seq_score[i + t.pairs] = static_cast<float>(score[1]);
        }
        if (t.drow != nullptr) {
            float g = t.reduction == GBCE_NONE ? t.grad_out[i] : t.grad_out[0];
            if (t.reduction == GBCE_MEAN)
                g /= static_cast<float>(t.pairs);
            s_d[0] = dh * weight[0] * g;
            s_d[1] = -dh * weight[1] * g;
        }
    }
    __syncthreads();
    if (t.drow != nullptr) {
        const float d = s_d[side];
        for (int64_t r = q.lo + first; r < q.hi; r += kHalf)
            t.drow[r] = preference_live(t, r) ? d : 0.0f;
    }
    __syncthreads();
    if (tid == 0) {
        __threadfence();  // this pair's outputs before the count
        if (bad)
            atomicOr(t.done, kBadOffsets);
        const int32_t before = atomicAdd(t.done, 1);
        s_last = (before & ~kBadOffsets) == static_cast<int32_t>(t.pairs) - 1;
        s_bad = bad || (before & kBadOffsets) != 0;
    }
    __syncthreads();
    if (!s_last)
        return;
    __threadfence();
    if (s_bad) {
        // Every step between two offsets was looked at by the pair it belongs to.  Where
        // one goes down or leaves the rows, sequences may share rows, and no pair's
        // scores or rows are its own.
        for (int64_t j = tid; j < 2 * t.pairs; j += kPairThreads) {
            if (j < t.pairs)
                t.loss_pairs[j] = kQuietNan;
            if (t.seq_score != nullptr)
                t.seq_score[j] = kQuietNan;
        }
        if (t.drow != nullptr) {
            const int64_t lo = t.offsets[0], hi = t.offsets[2 * t.pairs];
            for (int64_t r = tid; r < t.rows; r += kPairThreads)
                t.drow[r] = r >= lo && r < hi && preference_live(t, r) ? kQuietNan : 0.0f;
        }
        if (t.loss_out != nullptr && tid == 0)
            *t.loss_out = kQuietNan;
        return;
    }
    if (t.loss_out != nullptr) {
        s = Sum2{};
        n = 0;
        for (int64_t j = tid; j < t.pairs; j += kPairThreads)
            s.add(__ldcg(t.loss_pairs + j));
        cta_sum(s, n, scratch, counts);
        if (tid == 0)
            *t.loss_out = reduced(s, t.reduction == GBCE_MEAN, t.pairs);
    }
}

cudaError_t launch_pairs(const PreferenceTerms &t, cudaStream_t stream)
{
    const PostLaunch l(t.pairs, kPairThreads, 0, 1, stream);
    const cudaError_t err = cudaLaunchKernelEx(&l.cfg, preference_pair_kernel, t);
    note_launches(1);
    return err != cudaSuccess ? err : cudaGetLastError();
}

// Zeros for the rows of no sequence (a preference call from log-probs), and
// for the count of pairs done.
__global__ void __launch_bounds__(256)
    preference_outside_kernel(int64_t rows, const int64_t *offsets, int64_t sequences, float *drow,
                              int32_t *zero_out)
{
    const int64_t r = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (r == 0)
        *zero_out = 0;
    if (drow != nullptr && r < rows && (r < offsets[0] || r >= offsets[sequences]))
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
                         int64_t row_stride, double temperature)
{
    if (dtype != GBCE_F32 && dtype != GBCE_BF16)
        return GBCE_EDTYPE;
    if (rows < 0 || rows > kMaxRows || vocab < 1 || vocab > kMaxVocab || row_stride < vocab)
        return GBCE_EINVAL;
    if (!(temperature >= 1e-30 && temperature <= 1e30))
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

// v > 0 as hi + lo, hi of 14 bits, both positive: a logit of -inf times either
// part is -inf, where a lo of 0 or below would make its exponent NaN.
void two_floats(double v, float &hi, float &lo)
{
    int exponent = 0;
    const double mantissa = std::frexp(v, &exponent);
    hi = static_cast<float>(std::ldexp(std::floor(std::ldexp(mantissa, 14)), exponent - 14));
    lo = static_cast<float>(v - static_cast<double>(hi));
    if (!(lo > 0.0f))
        lo = hi * 0x1p-60f > 0.0f ? hi * 0x1p-60f : 0x1p-149f;
}

PostParams post_params(const void *logits, int64_t rows, int64_t vocab, int64_t row_stride,
                       double temperature, int32_t *dev_status)
{
    const double c = 1.4426950408889634 / temperature, it = 1.0 / temperature;
    PostParams p{};
    p.logits = logits;
    p.rows = rows;
    p.vocab = vocab;
    p.row_stride = row_stride;
    two_floats(c, p.c_hi, p.c_lo);
    two_floats(it, p.it_hi, p.it_lo);
    const double far = 0x1p31 / c;
    p.far = far < FLT_MAX ? static_cast<float>(far) : HUGE_VALF;
    p.k = 1;
    p.splits = 1;
    p.keep_from = INT64_MAX;
    p.dev_status = dev_status;
    return p;
}

cudaError_t launch_post(const PostParams &p, gbce_dtype dt, int op, int pass, cudaStream_t s)
{
    return dt == GBCE_BF16 ? gbce::launch_post<__nv_bfloat16>(p, op, pass, s)
                           : gbce::launch_post<float>(p, op, pass, s);
}

// Workspace of the calls with one loss per row: the item count (8 bytes), the
// row ticket, then at 256 [rows] floats of losses (or 16 bytes for each of the
// at most rows / 4096 + 1 parts of a long vector of log-probs).
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
    return n_items_out != nullptr ? gbce::launch_count_mask(nullptr, 0, n_items_out, nullptr, s)
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
    t.half_over_beta = 0.5 / static_cast<double>(o->beta);
    t.eps = o->label_smoothing;
    t.squared = o->kind == GBCE_PREFERENCE_SQUARED;
    t.average = o->average != 0;
}

struct PreferenceLayout {
    size_t loss, state, logp, grad, total;
};

PreferenceLayout preference_layout(int64_t rows, int64_t pairs)
{
    const size_t r = static_cast<size_t>(rows), n = static_cast<size_t>(pairs);
    PreferenceLayout w{};
    w.loss = 256;  // (the two sweeps' row tickets before it)
    w.state = w.loss + align_up(n * sizeof(float), 256);
    w.logp = w.state + align_up(2 * r * sizeof(float), 256);
    w.grad = w.logp + align_up(r * sizeof(float), 256);
    w.total = w.grad + align_up(r * sizeof(float), 256);
    return w;
}

constexpr int64_t kMaxPairs = int64_t(1) << 30;

}  // namespace

extern "C" {

// -------------------------------------------------------------- distillation

gbce_status distill_fwd(const void *logits, gbce_dtype dtype, int64_t rows, int64_t vocab,
                        int64_t row_stride, const int64_t *index, int64_t k,
                        const float *teacher_logits, const float *teacher_rest, double temperature,
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
    p.ticket = ws_at<int32_t>(workspace, 8);
    p.n_items_out = n_ptr;
    cudaError_t e = launch_post(p, dtype, gbce::kOpDistill, gbce::kPassFwd, s);
    if (e == cudaSuccess && reduction != GBCE_NONE)
        e = gbce::launch_sum_rows(p.loss_rows, rows, reduction == GBCE_MEAN, n_ptr, loss_out, s);
    return cuda_status(e);
}

gbce_status distill_bwd(const void *logits, gbce_dtype dtype, int64_t rows, int64_t vocab,
                        int64_t row_stride, const int64_t *index, int64_t k,
                        const float *teacher_logits, const float *teacher_rest, double temperature,
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
    p.dlogits = dlogits;
    p.d_stride = dlogits_row_stride;
    return cuda_status(launch_post(p, dtype, gbce::kOpDistill, gbce::kPassBwd,
                                   static_cast<cudaStream_t>(stream)));
}

gbce_status distill_fwd_bwd_fused(const void *logits, gbce_dtype dtype, int64_t rows,
                                  int64_t vocab, int64_t row_stride, const int64_t *index,
                                  int64_t k, const float *teacher_logits,
                                  const float *teacher_rest, double temperature,
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
    p.dlogits = dlogits;
    p.d_stride = dlogits_row_stride;
    p.ticket = ws_at<int32_t>(workspace, 8);
    p.n_items_out = n_ptr;
    cudaError_t e = launch_post(p, dtype, gbce::kOpDistill, gbce::kPassFused, s);
    if (e == cudaSuccess && reduction != GBCE_NONE)
        e = gbce::launch_sum_rows(p.loss_rows, rows, reduction == GBCE_MEAN, n_ptr, loss_out, s);
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
    gbce::PolicyRows q{};
    q.logp = logp;
    q.rows = rows;
    q.mask = row_mask;
    q.terms = policy_terms(options, advantages, old_logp, ref_logp);
    q.reduction = static_cast<int>(reduction);
    q.grad_out = grad_out;
    q.loss_rows = reduction == GBCE_NONE ? loss_out : nullptr;
    q.loss_out = loss_out;
    q.dlogp = dlogp_out;
    q.n_items = n_items_out != nullptr ? n_items_out : ws_at<int64_t>(workspace, 0);
    return cuda_status(gbce::launch_policy_rows(q, ws_at<void>(workspace, 256), s));
}

gbce_status policy_loss_fwd_bwd_fused(const void *logits, gbce_dtype dtype, int64_t rows,
                                      int64_t vocab, int64_t row_stride, const int64_t *labels,
                                      int64_t ignore_index, double temperature,
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
    p.dlogits = dlogits;
    p.d_stride = dlogits_row_stride;
    p.ticket = ws_at<int32_t>(workspace, 8);
    p.n_items_out = n_ptr;
    cudaError_t e = launch_post(p, dtype, gbce::kOpPolicy, gbce::kPassFused, s);
    if (e == cudaSuccess && reduction != GBCE_NONE)
        e = gbce::launch_sum_rows(p.loss_rows, rows, reduction == GBCE_MEAN, n_ptr, loss_out, s);
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
    const PreferenceLayout w = preference_layout(rows, pairs);
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
    t.loss_pairs = reduction == GBCE_NONE ? loss_out : ws_at<float>(workspace, w.loss);
    t.loss_out = reduction == GBCE_NONE ? nullptr : loss_out;
    t.done = ws_at<int32_t>(workspace, 64);
    t.seq_score = seq_score_out;
    t.drow = dlogp_out;
    t.dev_status = dev_status;
    const int64_t outside = dlogp_out != nullptr && rows > 0 ? (rows + 255) / 256 : 1;
    gbce::preference_outside_kernel<<<static_cast<unsigned>(outside), 256, 0, s>>>(
        rows, seq_offsets, 2 * pairs, dlogp_out, t.done);
    gbce::note_launches(1);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess)
        e = gbce::launch_pairs(t, s);
    return cuda_status(e);
}

gbce_status preference_loss_fwd_bwd_fused(
    const void *logits, gbce_dtype dtype, int64_t rows, int64_t vocab, int64_t row_stride,
    const int64_t *labels, int64_t ignore_index, double temperature, const int64_t *seq_offsets,
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
    float *logp = logp_out != nullptr ? logp_out : ws_at<float>(workspace, w.logp);
    float *grad = ws_at<float>(workspace, w.grad);
    float *state = ws_at<float>(workspace, w.state);
    cudaError_t e = cudaSuccess;
    PostParams p = post_params(logits, rows, vocab, row_stride, temperature, dev_status);
    p.labels = labels;
    p.ignore_index = ignore_index;
    p.row_range = seq_offsets;
    p.row_range_end = 2 * pairs;
    if (rows > 0) {
        // log p and the rest's state of every row of a sequence
        p.logp_out = logp;
        p.rest_state_out = state;
        p.ticket = ws_at<int32_t>(workspace, 0);
        p.zero_out = ws_at<int32_t>(workspace, 64);
        // the last rows stay in L2 (with all of them marked to stay, a batch that
        // exceeds L2 loses 2% to its own rows' evictions)
        const int64_t row = vocab * static_cast<int64_t>(elem_size(dtype));
        const int64_t fit = (int64_t(96) << 20) / row;
        p.keep_from = rows > fit ? rows - fit : 0;
        e = launch_post(p, dtype, gbce::kOpToken, gbce::kPassFwd, s);
    } else {
        e = cudaMemsetAsync(workspace, 0, 256, s);
    }
    PreferenceTerms t{};
    t.logp = logp;
    t.ref_logp = ref_logp;
    t.rows = rows;
    t.pairs = pairs;
    t.offsets = seq_offsets;
    t.labels = labels;
    t.ignore_index = ignore_index;
    set_preference_options(t, options);
    t.reduction = static_cast<int>(reduction);
    t.grad_out = grad_out;
    t.loss_pairs = reduction == GBCE_NONE ? loss_out : ws_at<float>(workspace, w.loss);
    t.loss_out = reduction == GBCE_NONE ? nullptr : loss_out;
    t.done = ws_at<int32_t>(workspace, 64);
    t.seq_score = seq_score_out;
    t.drow = grad;
    t.dev_status = dev_status;
    if (e == cudaSuccess)
        e = gbce::launch_pairs(t, s);
    if (e == cudaSuccess && rows > 0) {
        // the rows that were read last are in L2 still: they come first
        p.logp_out = nullptr;
        p.rest_state_out = nullptr;
        p.rest_state = state;
        p.grad_out = grad;
        p.reduction = GBCE_NONE;
        p.ticket = ws_at<int32_t>(workspace, 128);
        p.zero_out = nullptr;
        p.keep_from = INT64_MAX;
        p.reverse = 1;
        p.dlogits = dlogits;
        p.d_stride = dlogits_row_stride;
        e = launch_post(p, dtype, gbce::kOpToken, gbce::kPassBwd, s);
    }
    return cuda_status(e);
}

}  // extern "C"
