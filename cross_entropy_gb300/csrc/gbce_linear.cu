// Row selection, packing, and the per-row steps around the products of the
// calls that start from hidden states (see gbce_linear.h).
#include "gbce_kernels.cuh"
#include "gbce_linear.h"
#include "gbce_linear_rows.cuh"

namespace gbce {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

__device__ __forceinline__ float nan_value() { return __int_as_float(0x7fc00000); }

}  // namespace

// Whether row r takes part (`live`) and counts (`item`: it was not masked or
// ignored, though its target may be out of range).
__device__ __forceinline__ void row_kind(const LinParams &p, int64_t r, bool &live, bool &item)
{
    const int K = static_cast<int>(p.k);
    const bool masked = p.row_mask != nullptr && p.row_mask[r] == 0;
    item = !masked && !(p.token_ce && p.targets[r] == p.ignore_index);
    live = item;
    if (item && (p.token_ce || p.whole_rows))
        for (int k = 0; k < K; ++k) {
            const int64_t t = p.targets[r * K + k];
            live = live && t >= 0 && t < p.vocab;
        }
}

// Forward outputs and the map entry of a row that takes no part.
__device__ __forceinline__ void leave_out(const LinParams &p, int64_t r, bool item)
{
    const int K = static_cast<int>(p.k);
    const float fill = item ? nan_value() : 0.0f;
    if (item)
        report(p.dev_status, p.token_ce ? GBCE_DEV_BAD_LABEL : GBCE_DEV_BAD_INDEX);
    p.row_map[r] = item ? kLinRowBad : kLinRowSkipped;
    if (p.logp_out != nullptr)
        for (int k = 0; k < K; ++k)
            p.logp_out[r * K + k] = fill;
    if (p.state_out != nullptr) {
        p.state_out[2 * r] = item ? fill : kNegInf;
        p.state_out[2 * r + 1] = fill;
    }
    if (p.loss_rows != nullptr)
        p.loss_rows[r] = fill;
}

// The factor of both gradients that every row shares: a summed or averaged
// loss's upstream gradient over T (and the number of items).  It stays out of
// dz and joins at the end, in fp32, so that it is not rounded with each dz.
__device__ __forceinline__ float shared_factor(const LinParams &p)
{
    if (!p.token_ce || p.reduction == 0)
        return 1.0f;
    double a = static_cast<double>(p.grad_out[0]) / static_cast<double>(p.T);
    if (p.reduction == 2) {
        const int64_t n = p.n_items != nullptr ? *p.n_items : p.head->n_items;
        a = n > 0 ? a / static_cast<double>(n) : 0.0;
    }
    return static_cast<float>(a);
}

// What the CE gradient of packed row i takes besides its logits: (M, u / S)
// for the p_j and the label's u expm1(log p), which keeps 1 - p when p rounds
// to 1; u = upstream / T where rows have their own.
__device__ __forceinline__ void ce_row_gradient(const LinParams &p, int64_t i, int64_t r, float M,
                                                float S, float logp)
{
    const float u = p.reduction == 0 ? p.grad_out[r] * (1.0f / p.T) : 1.0f;
    p.grow[i] = make_float2(M, u / S);
    p.dzt[i] = u * expm1f(logp);
}

// A backward call's row, from the forward's log-probs and row state; thread k
// of the CTA has target k.  The selective gradient has (M, -G / (T S)) and, for
// a gathered column,
//   (-g_t expm1(log p_t) - (sum of the others' g) p_t) / T.
__device__ __forceinline__ void saved_row_gradient(const LinParams &p, int64_t i, int64_t r)
{
    const int K = static_cast<int>(p.k), k = static_cast<int>(threadIdx.x);
    if (k >= K)
        return;
    const float M = p.saved_state[2 * r], S = p.saved_state[2 * r + 1];
    const float logp = p.saved_logp[r * K + k];
    if (p.token_ce) {
        ce_row_gradient(p, i, r, M, S, logp);
        return;
    }
    // sums of upstream in fp64 (in fp32 one that cancels keeps only its terms'
    // rounding), the others' from their own terms rather than as a difference,
    // and over T before they meet the probabilities
    const float *g = p.grad_out + r * K;
    const int64_t *t = p.targets + r * K;
    const int64_t own = t[k];
    double sum = 0.0, mine = 0.0, other = 0.0;
    for (int j = 0; j < K; ++j) {
        const double gj = g[j];
        sum += gj;
        if (t[j] == own)
            mine += gj;
        else
            other += gj;
    }
    if (k == 0)
        p.grow[i] = make_float2(M, -static_cast<float>(sum / p.T) / S);
    p.dzt[i * K + k] = fmaf(-static_cast<float>(mine / p.T), expm1f(logp),
                            -static_cast<float>(other / p.T) * expf(logp));
}

__device__ __forceinline__ void write_head(const LinParams &p, int32_t live, int64_t items)
{
    p.head->n_live = live;
    p.head->n_items = items;
    p.head->alpha = p.backward && !p.fused ? shared_factor(p) : 1.0f;
    p.head->done = 0;
    if (p.n_items_out != nullptr)
        *p.n_items_out = items;
}

// Which rows take part, as a stable partition: row_list[i] is the i-th live
// row, row_map[r] its place or why it has none.  One CTA: it reads rows x
// (k + 1) words, 1024 rows per step by warp ballots and a scan over the warps;
// every later kernel depends on its count.
__global__ void __launch_bounds__(kPlanThreads) lin_plan_kernel(LinParams p)
{
    __shared__ int32_t s_live[kPlanWarps], s_item[kPlanWarps];
    grid_dependency_wait();
    launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t base = 0;
    int64_t items = 0;
    for (int64_t r0 = 0; r0 < p.rows; r0 += kPlanThreads) {
        const int64_t r = r0 + threadIdx.x;
        bool live = false, item = false;
        if (r < p.rows) {
            row_kind(p, r, live, item);
            if (!live)
                leave_out(p, r, item);
        }
        const unsigned bl = __ballot_sync(0xffffffffu, live);
        const unsigned bi = __ballot_sync(0xffffffffu, item);
        if (lane == 0) {
            s_live[warp] = __popc(bl);
            s_item[warp] = __popc(bi);
        }
        __syncthreads();
        int32_t before = 0, total = 0, titem = 0;
#pragma unroll
        for (int w = 0; w < kPlanWarps; ++w) {
            before += w < warp ? s_live[w] : 0;
            total += s_live[w];
            titem += s_item[w];
        }
        if (live) {
            const int32_t i = base + before + __popc(bl & ((1u << lane) - 1u));
            p.row_list[i] = static_cast<int32_t>(r);
            p.row_map[r] = i;
        }
        base += total;
        items += titem;
        __syncthreads();  // before the next step overwrites the counts
    }
    if (threadIdx.x == 0)
        write_head(p, base, items);
}

// Four elements at a time.
template <typename T> struct Quad;
template <> struct Quad<__nv_bfloat16> { using type = uint2; };
template <> struct Quad<float> { using type = float4; };

// Eight values into their planes: bf16 x is its own; fp32 x = hi + mid + lo,
// each the rounding of what is left (24 bits in three times 8).
template <int PLANES>
__device__ __forceinline__ void store_eight(float (&x)[8], __nv_bfloat16 *dst, int64_t plane)
{
#pragma unroll
    for (int z = 0; z < PLANES; ++z) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = float2_to_bf16x2(make_float2(x[2 * i], x[2 * i + 1]));
            const float2 f = bf16x2_to_float2(w[i]);
            x[2 * i] -= f.x;
            x[2 * i + 1] -= f.y;
        }
        *reinterpret_cast<uint4 *>(dst + z * plane) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Elements [d, d + 8) of a row into its planes, whose rows start on 16 bytes;
// past the row's end its padding takes the rest.
template <typename T, int PLANES>
__device__ __forceinline__ void pack_eight(const T *src, __nv_bfloat16 *dst, int64_t plane, int64_t d,
                                           int64_t dim, bool zero)
{
    float x[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (!zero)
        read_eight(src, d, dim, x);
    store_eight<PLANES>(x, dst + d, plane);
}

// Packed row i from row r of the hidden states (zeros past the live rows), its
// targets, their logits where there are many, and in a backward call what its
// gradient takes.
template <typename T, int PLANES>
__device__ __forceinline__ void pack_hidden(const LinParams &p, int64_t i, int64_t r, bool in)
{
    const T *src = static_cast<const T *>(p.hidden) + r * p.hidden_stride;
    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.hpack) + i * p.pitch;
    for (int64_t d = 8 * static_cast<int64_t>(threadIdx.x); d < p.dim; d += 8 * blockDim.x)
        pack_eight<T, PLANES>(src, dst, p.hpack_plane, d, p.dim, !in);
    const int K = static_cast<int>(p.k);
    for (int k = threadIdx.x; k < K; k += blockDim.x) {
        const int64_t t = in ? p.targets[r * K + k] : -1;
        p.tgt[i * K + k] = t >= 0 && t < p.vocab ? static_cast<int32_t>(t) : -1;
    }
    if (in && lin_dots_in_pack(p))
        for (int k = threadIdx.x >> 5; k < K; k += blockDim.x >> 5) {
            const int64_t t = p.targets[r * K + k];
            if (t < 0 || t >= p.vocab)
                continue;
            const float x = row_dot(src, static_cast<const T *>(p.weight) + t * p.weight_stride, p.dim);
            if ((threadIdx.x & 31) == 0)
                p.xt[i * K + k] = x;
        }
    if (in && p.backward && !p.fused)
        saved_row_gradient(p, i, r);
}

// Rows of a weight that the products cannot read in place (fp32, or rows that
// do not start on 16 bytes): rows [v0, v0 + rows) into the packed piece from
// its start, weight_rows_per_cta of them by CTA `cta`, enough to keep its
// threads busy when rows are short.
__host__ __device__ __forceinline__ int64_t weight_rows_per_cta(int64_t dim)
{
    return dim >= 2048 ? 1 : (dim <= 64 ? 32 : 2048 / dim);
}

template <typename T, int PLANES>
__device__ __forceinline__ void pack_weight(const LinParams &p, int64_t cta, int64_t v0, int64_t rows)
{
    const int64_t per = weight_rows_per_cta(p.dim), i0 = cta * per;
    const uint32_t parts = static_cast<uint32_t>((p.dim + 7) / 8);
    const uint32_t all = static_cast<uint32_t>(min(per, rows - i0)) * parts;
    for (uint32_t e = threadIdx.x; e < all; e += blockDim.x) {
        const int64_t i = i0 + e / parts;
        pack_eight<T, PLANES>(static_cast<const T *>(p.weight) + (v0 + i) * p.weight_stride,
                              static_cast<__nv_bfloat16 *>(p.wpack) + i * p.pitch, p.wpack_rows * p.pitch,
                              8 * static_cast<int64_t>(e % parts), p.dim, false);
    }
}

// One CTA per packed row.  A backward product over the rows reads whole
// 64-deep blocks of them: the rows up to the next multiple of kLinRowPad are
// zeros there.
template <typename T, int PLANES>
__global__ void __launch_bounds__(128) lin_pack_kernel(LinParams p)
{
    grid_dependency_wait();
    launch_dependents();
    const int32_t live = p.head->n_live;
    const int64_t i = blockIdx.x;
    if (i >= (static_cast<int64_t>(live) + kLinRowPad - 1) / kLinRowPad * kLinRowPad)
        return;
    pack_hidden<T, PLANES>(p, i, i < live ? p.row_list[i] : 0, i < live);
}

template <typename T, int PLANES>
__global__ void __launch_bounds__(128) lin_pack_weight_kernel(LinParams p, int64_t v0, int64_t rows)
{
    grid_dependency_wait();
    launch_dependents();
    pack_weight<T, PLANES>(p, blockIdx.x, v0, rows);
}

// Plan and packing in one launch, for calls of up to kSmallRows rows whose
// time is launches: every CTA finds its own row by counting all of them, the
// first writes the plan down.  CTAs from `packed` on pack the weight, where
// it needs that and fits whole.  (64 x 4096 x 256 fp32: three launches' 14
// us became one's 6.6.)
constexpr int kSmallRows = 1024, kSmallTargets = 4096;

template <typename T, int PLANES>
__global__ void __launch_bounds__(128) lin_small_pack_kernel(LinParams p, int32_t packed)
{
    __shared__ uint32_t s_live[kSmallRows / 32], s_item[kSmallRows / 32];
    __shared__ int32_t s_before[kSmallRows / 32], s_row, s_total;
    grid_dependency_wait();
    launch_dependents();
    if (blockIdx.x >= packed) {
        pack_weight<T, PLANES>(p, static_cast<int64_t>(blockIdx.x) - packed, 0, p.vocab);
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool first = blockIdx.x == 0;
#pragma unroll
    for (int it = 0; it < kSmallRows / 128; ++it) {
        const int r = it * 128 + static_cast<int>(threadIdx.x);
        bool live = false, item = false;
        if (r < p.rows) {
            row_kind(p, r, live, item);
            if (first && !live)
                leave_out(p, r, item);
        }
        const unsigned bl = __ballot_sync(0xffffffffu, live);
        const unsigned bi = __ballot_sync(0xffffffffu, item);
        if (lane == 0) {
            s_live[it * 4 + warp] = bl;
            s_item[it * 4 + warp] = bi;
        }
    }
    __syncthreads();
    if (warp == 0) {
        // lane l has rows [32 l, 32 l + 32); the i-th live row is in the word
        // whose running count passes i
        const uint32_t word = s_live[lane];
        int32_t upto = __popc(word), items = __popc(s_item[lane]);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t x = __shfl_up_sync(0xffffffffu, upto, o);
            upto += lane >= o ? x : 0;
        }
        items = __reduce_add_sync(0xffffffffu, items);
        const int32_t before = upto - __popc(word), i = static_cast<int32_t>(blockIdx.x);
        if (before <= i && i < upto) {
            uint32_t w = word;
            for (int32_t skip = i - before; skip > 0; --skip)
                w &= w - 1;
            s_row = lane * 32 + __ffs(w) - 1;
        }
        if (lane == 31)
            s_total = upto;
        s_before[lane] = before;
        if (first && lane == 31)
            write_head(p, upto, items);
    }
    __syncthreads();
    if (first) {
#pragma unroll
        for (int it = 0; it < kSmallRows / 128; ++it) {
            const uint32_t w = s_live[it * 4 + warp];
            const int32_t r = it * 128 + static_cast<int32_t>(threadIdx.x);
            const int32_t at = s_before[it * 4 + warp] + __popc(w & ((1u << lane) - 1u));
            if (w >> lane & 1u) {
                p.row_list[at] = r;
                p.row_map[r] = at;
            }
        }
    }
    const int32_t live = s_total;
    const int64_t i = blockIdx.x;
    if (i >= (static_cast<int64_t>(live) + kLinRowPad - 1) / kLinRowPad * kLinRowPad)
        return;
    pack_hidden<T, PLANES>(p, i, i < live ? s_row : 0, i < live);
}

// One gathered logit into a (max, sum).  A NaN stays one: merge_max_sum would
// take it for nothing where nothing else is (its max is then -inf).
__device__ __forceinline__ void add_logit(float &m, float &s, float x, float c)
{
    merge_max_sum(m, s, x, 1.0f, c);
    if (x != x) {
        m = m == kNegInf ? 0.0f : m;
        s = x;
    }
}

// One warp per live row: its tiles' partials merged in a fixed order (lane l
// takes the tiles l, l + 32, ..., eight at a time, then the lanes merge), then
// the log-probs of its targets, each over the other columns, and the whole
// row's state.  Lane k has target k; a target gathered before counts once.
// A direct call's rows were not selected: the warp finds out about its row
// here, and counts it.  The last CTA to finish sums the losses of all rows, in
// row order per thread and over the threads in a fixed tree: the order does
// not depend on which CTA that is.
constexpr int kCombineWarps = 4;

__global__ void __launch_bounds__(32 * kCombineWarps) lin_combine_kernel(LinParams p)
{
    __shared__ int32_t s_last;
    __shared__ double s_sum[kCombineWarps];
    grid_dependency_wait();
    launch_dependents();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kCombineWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int K = static_cast<int>(p.k);
    bool live = i < p.head->n_live;
    int64_t r = i;
    int32_t tg = -1;
    if (live && p.direct) {
        // nothing was selected or packed: this warp's row is sorted out here
        bool item;
        row_kind(p, r, live, item);
        if (lane == 0 && item && p.token_ce)
            atomicAdd(reinterpret_cast<unsigned long long *>(&p.head->n_items), 1ull);
        if (!live && lane == 0)
            leave_out(p, r, item);
        const int64_t t = lane < K ? p.targets[i * K + lane] : -1;
        tg = t >= 0 && t < p.vocab ? static_cast<int32_t>(t) : -1;
    } else if (live) {
        r = p.row_list[i];
        tg = lane < K ? p.tgt[i * K + lane] : -1;
    }
    if (live) {
        const float xt = lane < K ? p.xt[i * K + lane] : 0.0f;
        float m = kNegInf, s = 0.0f, unused = 0.0f;
        const float2 *part = p.partials + i * p.tiles;
        for (int64_t t0 = 0; t0 < p.tiles; t0 += 256) {
            float2 x[8];
            float top = m;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int64_t t = t0 + u * 32 + lane;
                x[u] = t < p.tiles ? part[t] : make_float2(kNegInf, 0.0f);
                top = fmaxf(top, x[u].x);
            }
            const float ref = top == kNegInf ? 0.0f : top;
            s *= ex2((m - ref) * p.c);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                s = fmaf(x[u].y, ex2((x[u].x - ref) * p.c), s);
            m = top;
        }
        warp_merge_state<0>(m, s, unused, p.c, 0.0f);
        // others of target k: (m, s) and the distinct targets that are not k
        const unsigned same = __match_any_sync(0xffffffffu, tg);
        const bool counts = tg >= 0 && (same & ((1u << lane) - 1u)) == 0;
        float om = m, os = s, M = m, S = s;
        for (int j = 0; j < K; ++j) {
            const int32_t tj = __shfl_sync(0xffffffffu, tg, j);
            const float xj = __shfl_sync(0xffffffffu, xt, j);
            if (__shfl_sync(0xffffffffu, static_cast<int>(counts), j) == 0)
                continue;
            add_logit(M, S, xj, p.c);
            if (tj != tg)
                add_logit(om, os, xj, p.c);
        }
        float logp = 0.0f;
        if (lane < K) {
            logp = nan_value();
            if (tg < 0)
                report(p.dev_status, GBCE_DEV_BAD_INDEX);
            else
                logp = finalize_logp(om, os, xt, p.T);
            if (p.logp_out != nullptr)
                p.logp_out[r * K + lane] = logp;
        }
        if (lane == 0) {
            if (p.loss_rows != nullptr)
                p.loss_rows[r] = -logp;
            if (p.state_out != nullptr) {
                p.state_out[2 * r] = M;
                p.state_out[2 * r + 1] = S;
            }
            if (p.fused)
                ce_row_gradient(p, i, r, M, S, logp);
        }
    }
    if (p.fused && blockIdx.x == 0 && threadIdx.x == 0)
        p.head->alpha = shared_factor(p);
    if (p.loss_out == nullptr && !(p.direct && p.n_items_out != nullptr))
        return;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0)
        s_last = atomicAdd(&p.head->done, 1) == static_cast<int32_t>(gridDim.x) - 1;
    __syncthreads();
    if (!s_last)
        return;
    __threadfence();
    const int64_t n = *reinterpret_cast<volatile int64_t *>(&p.head->n_items);
    if (p.direct && threadIdx.x == 0 && p.n_items_out != nullptr)
        *p.n_items_out = n;
    if (p.loss_out == nullptr)
        return;
    double sum = 0.0;
    for (r = threadIdx.x; r < p.rows; r += 32 * kCombineWarps)
        sum += static_cast<double>(__ldcg(p.loss_rows + r));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0)
        s_sum[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        double total = 0.0;
        for (int w = 0; w < kCombineWarps; ++w)
            total += s_sum[w];
        *p.loss_out = static_cast<float>(p.reduction == 2 ? (n > 0 ? total / static_cast<double>(n) : 0.0) : total);
    }
}

// dz from kept logits (a fused CE call): one CTA per packed row and stretch of
// kDzSpan columns; rows up to the next 64 and columns up to the next 64 are
// zeros, which the products read.  Bound by memory: 4 bytes of logit and 2 (6
// for fp32 inputs) of dz a column.
constexpr int kDzThreads = 128, kDzSpan = kDzThreads * 8 * 4;

template <int PLANES> __global__ void __launch_bounds__(kDzThreads) lin_dz_kernel(LinParams p)
{
    grid_dependency_wait();
    launch_dependents();
    const int32_t live = p.head->n_live;
    const int64_t i = blockIdx.x;
    if (i >= (static_cast<int64_t>(live) + 63) / 64 * 64)
        return;
    const bool in = i < live;
    const float2 g = in ? p.grow[i] : make_float2(0.0f, 0.0f);
    const int64_t t = in ? p.tgt[i] : -1;
    const float dzt = in ? p.dzt[i] : 0.0f;
    const int64_t end = (p.vocab + 63) / 64 * 64;
    const float *z = p.z + i * p.piece;
    __nv_bfloat16 *dz = static_cast<__nv_bfloat16 *>(p.dz) + i * p.piece;
    const int64_t c0 = static_cast<int64_t>(blockIdx.y) * kDzSpan + threadIdx.x * 8;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t c = c0 + u * kDzThreads * 8;
        if (c >= end)
            return;
        float x[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (in) {
            load_eight(z + c, true, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = c + j < p.vocab ? g.y * ex2((x[j] - g.x) * p.c) : 0.0f;
                x[j] = c + j == t ? dzt : x[j];
            }
        }
        store_eight<PLANES>(x, dz + c, p.dz_plane);
    }
}

// dhidden by original row: alpha times the sum of its parts, zeros for rows
// left out, NaN for rows with a target out of range.  Four values a thread.
template <typename T>
__global__ void __launch_bounds__(128) lin_finish_kernel(LinParams p)
{
    grid_dependency_wait();
    launch_dependents();
    const int64_t r = blockIdx.x;
    const int32_t i = p.row_map[r], parts = p.head->dh_splits;
    const int32_t m = 128 * p.grads_tile.ctas;
    const int64_t part = static_cast<int64_t>((p.head->n_live + m - 1) / m) * m * p.dh_pitch;
    const float alpha = p.head->alpha;
    T *out = static_cast<T *>(p.dhidden) + r * p.dhidden_stride;
    const bool quads = reinterpret_cast<uintptr_t>(p.dhidden) % (4 * sizeof(T)) == 0 && p.dhidden_stride % 4 == 0;
    const float fill = i == kLinRowBad ? nan_value() : 0.0f;
    const float *sums = p.dh + (i >= 0 ? i : 0) * p.dh_pitch;
    for (int64_t d = 4 * static_cast<int64_t>(threadIdx.x); d < p.dim; d += 4 * blockDim.x) {
        float4 x = make_float4(fill, fill, fill, fill);
        if (i >= 0) {
            x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
            for (int z = 0; z < parts; ++z) {
                const float4 y = *reinterpret_cast<const float4 *>(sums + z * part + d);
                x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
            }
            x = make_float4(alpha * x.x, alpha * x.y, alpha * x.z, alpha * x.w);
        }
        const float f[4] = {x.x, x.y, x.z, x.w};
        if (quads && d + 4 <= p.dim) {
            typename Quad<T>::type w;
            T *e = reinterpret_cast<T *>(&w);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                e[j] = T(f[j]);
            *reinterpret_cast<typename Quad<T>::type *>(out + d) = w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (d + j < p.dim)
                    out[d + j] = T(f[j]);
        }
    }
}

// ---------------------------------------------------------------- launches

namespace {

// Launch as a programmatic dependent of the kernel before it on the stream.
template <typename... Args>
cudaError_t launch_after(void (*kernel)(Args...), dim3 grid, dim3 block, size_t smem,
                         cudaStream_t s, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    note_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

unsigned blocks(int64_t n, int64_t per) { return static_cast<unsigned>((n + per - 1) / per); }

}  // namespace

cudaError_t lin_select(const LinParams &p, cudaStream_t s)
{
    if (p.direct)
        return cudaSuccess;
    const int64_t packed = p.backward ? p.rows_pad : p.rows;
    if (p.rows <= kSmallRows && p.rows * p.k <= kSmallTargets) {
        const int64_t weight = p.weight_direct || p.wpack_rows < p.vocab
                                   ? 0
                                   : blocks(p.vocab, weight_rows_per_cta(p.dim));
        return launch_after(p.bf16 ? lin_small_pack_kernel<__nv_bfloat16, 1> : lin_small_pack_kernel<float, 3>,
                            dim3(static_cast<unsigned>(packed + weight)), dim3(128), 0, s, p,
                            static_cast<int32_t>(packed));
    }
    const cudaError_t e = launch_after(lin_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, p);
    return e != cudaSuccess
               ? e
               : launch_after(p.bf16 ? lin_pack_kernel<__nv_bfloat16, 1> : lin_pack_kernel<float, 3>,
                              dim3(static_cast<unsigned>(packed)), dim3(128), 0, s, p);
}

bool lin_weight_packed(const LinParams &p)
{
    return !p.direct && !p.weight_direct && p.wpack_rows >= p.vocab && p.rows <= kSmallRows &&
           p.rows * p.k <= kSmallTargets;
}

cudaError_t lin_pack_weight(const LinParams &p, int64_t v0, int64_t v1, cudaStream_t s)
{
    return launch_after(p.bf16 ? lin_pack_weight_kernel<__nv_bfloat16, 1>
                               : lin_pack_weight_kernel<float, 3>,
                        dim3(blocks(v1 - v0, weight_rows_per_cta(p.dim))), dim3(128), 0, s, p, v0, v1 - v0);
}

cudaError_t lin_combine(const LinParams &p, cudaStream_t s)
{
    return launch_after(lin_combine_kernel, dim3(blocks(p.rows, kCombineWarps)), dim3(32 * kCombineWarps), 0,
                        s, p);
}

cudaError_t lin_dz(const LinParams &p, cudaStream_t s)
{
    const int64_t columns = (p.vocab + 63) / 64 * 64;
    return launch_after(p.planes == 1 ? lin_dz_kernel<1> : lin_dz_kernel<3>,
                        dim3(blocks(p.rows, 64) * 64, blocks(columns, kDzSpan)), dim3(kDzThreads), 0,
                        s, p);
}

cudaError_t lin_finish(const LinParams &p, cudaStream_t s)
{
    return launch_after(p.bf16 ? lin_finish_kernel<__nv_bfloat16> : lin_finish_kernel<float>,
                        dim3(static_cast<unsigned>(p.rows)), dim3(128), 0, s, p);
}

}  // namespace gbce
