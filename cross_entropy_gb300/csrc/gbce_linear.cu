// Row selection, packing, and the per-row steps around the products of the
// calls that start from hidden states (see gbce_linear.h).
#include "gbce_kernels.cuh"
#include "gbce_linear.h"

namespace gbce {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

__device__ __forceinline__ float nan_value() { return __int_as_float(0x7fc00000); }

}  // namespace

// Which rows take part, as a stable partition: row_list[i] is the i-th live
// row, row_map[r] its place or why it has none.  Rows that take no part get
// their forward outputs here (0, or NaN for a target out of range).  One CTA:
// it reads rows x (k + 1) words, 1024 rows per step by warp ballots and a
// scan over the warps; every later kernel depends on its count.
__global__ void __launch_bounds__(kPlanThreads) lin_plan_kernel(LinParams p)
{
    __shared__ int32_t s_live[kPlanWarps], s_item[kPlanWarps];
    launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int K = static_cast<int>(p.k);
    int32_t base = 0;
    int64_t items = 0;
    for (int64_t r0 = 0; r0 < p.rows; r0 += kPlanThreads) {
        const int64_t r = r0 + threadIdx.x;
        bool live = false, item = false;
        if (r < p.rows) {
            const bool masked = p.row_mask != nullptr && p.row_mask[r] == 0;
            item = !masked && !(p.token_ce && p.targets[r] == p.ignore_index);
            live = item;
            if (item && (p.token_ce || p.whole_rows)) {
                for (int k = 0; k < K; ++k) {
                    const int64_t t = p.targets[r * K + k];
                    live = live && t >= 0 && t < p.vocab;
                }
                if (!live)
                    report(p.dev_status, p.token_ce ? GBCE_DEV_BAD_LABEL : GBCE_DEV_BAD_INDEX);
            }
            if (!live) {
                const float fill = item ? nan_value() : 0.0f;
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
    if (threadIdx.x == 0) {
        p.head->n_live = base;
        p.head->n_items = items;
        p.head->alpha = 1.0f;
        if (p.n_items_out != nullptr)
            *p.n_items_out = items;
    }
}

// Four elements at a time, or one.
template <typename T> struct Quad;
template <> struct Quad<__nv_bfloat16> { using type = uint2; };
template <> struct Quad<float> { using type = float4; };

// Planes of a value: bf16 x is its own; fp32 x = hi + mid + lo, each the
// rounding of what is left (24 bits in three times 8).
template <int PLANES>
__device__ __forceinline__ void store_planes(float x, __nv_bfloat16 *dst, int64_t plane)
{
#pragma unroll
    for (int z = 0; z < PLANES; ++z) {
        const __nv_bfloat16 w = __float2bfloat16_rn(x);
        dst[z * plane] = w;
        x -= __bfloat162float(w);
    }
}

// One row of an operand into its planes; `quads` when both sides allow four
// elements at a time.
template <typename T, int PLANES>
__device__ __forceinline__ void pack_row(const T *src, __nv_bfloat16 *dst, int64_t plane,
                                         int64_t dim, bool quads, bool zero)
{
    int64_t done = 0;
    if (quads) {
        done = dim / 4 * 4;
        for (int64_t d = 4 * static_cast<int64_t>(threadIdx.x); d < done; d += 4 * blockDim.x) {
            float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (!zero) {
                const auto raw = *reinterpret_cast<const typename Quad<T>::type *>(src + d);
                const T *e = reinterpret_cast<const T *>(&raw);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[i] = static_cast<float>(e[i]);
            }
#pragma unroll
            for (int z = 0; z < PLANES; ++z) {
                uint2 w;
                w.x = float2_to_bf16x2(make_float2(x[0], x[1]));
                w.y = float2_to_bf16x2(make_float2(x[2], x[3]));
                *reinterpret_cast<uint2 *>(dst + z * plane + d) = w;
                const float2 lo = bf16x2_to_float2(w.x), hi = bf16x2_to_float2(w.y);
                x[0] -= lo.x;
                x[1] -= lo.y;
                x[2] -= hi.x;
                x[3] -= hi.y;
            }
        }
    }
    for (int64_t d = done + threadIdx.x; d < dim; d += blockDim.x)
        store_planes<PLANES>(zero ? 0.0f : static_cast<float>(src[d]), dst + d, plane);
}

template <typename T>
__device__ __forceinline__ bool quad_rows(const T *base, int64_t stride)
{
    constexpr uint64_t bytes = 4 * sizeof(T);
    return reinterpret_cast<uintptr_t>(base) % bytes == 0 && stride % 4 == 0;
}

// Packed hidden states and targets of the live rows, one CTA per packed row;
// the rows up to the next multiple of kLinRowPad are zeros.
template <typename T, int PLANES>
__global__ void __launch_bounds__(128) lin_pack_kernel(LinParams p)
{
    grid_dependency_wait();
    launch_dependents();
    const int32_t live = p.head->n_live;
    const int64_t i = blockIdx.x;
    if (i >= (static_cast<int64_t>(live) + kLinRowPad - 1) / kLinRowPad * kLinRowPad)
        return;
    const bool in = i < live;
    const int64_t r = in ? p.row_list[i] : 0;
    const T *base = static_cast<const T *>(p.hidden);
    pack_row<T, PLANES>(base + r * p.hidden_stride, static_cast<__nv_bfloat16 *>(p.hpack) + i * p.pitch,
                        p.hpack_plane, p.dim, quad_rows(base, p.hidden_stride), !in);
    const int K = static_cast<int>(p.k);
    for (int k = threadIdx.x; k < K; k += blockDim.x) {
        const int64_t t = in ? p.targets[r * K + k] : -1;
        p.tgt[i * K + k] = t >= 0 && t < p.vocab ? static_cast<int32_t>(t) : -1;
    }
}

// One piece of a weight that the products cannot read in place: fp32, or rows
// that do not start on 16 bytes.
template <typename T, int PLANES>
__global__ void __launch_bounds__(128) lin_pack_weight_kernel(LinParams p, int64_t v0)
{
    grid_dependency_wait();
    launch_dependents();
    const int64_t i = blockIdx.x;
    const T *base = static_cast<const T *>(p.weight);
    pack_row<T, PLANES>(base + (v0 + i) * p.weight_stride,
                        static_cast<__nv_bfloat16 *>(p.wpack) + i * p.pitch, p.wpack_rows * p.pitch,
                        p.dim, quad_rows(base, p.weight_stride), false);
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

// One warp per live row: its tiles' partials merged in a fixed order (lane l
// takes the tiles l, l + 32, ..., then the lanes merge), then the log-probs
// of its targets, each over the other columns, and the whole row's state.
__global__ void __launch_bounds__(128) lin_combine_kernel(LinParams p)
{
    grid_dependency_wait();
    launch_dependents();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (i >= p.head->n_live)
        return;
    const int lane = threadIdx.x & 31;
    const int K = static_cast<int>(p.k);
    float m = kNegInf, s = 0.0f, unused = 0.0f;
    for (int64_t t = lane; t < p.tiles; t += 32) {
        const float2 part = p.partials[i * p.tiles + t];
        merge_max_sum(m, s, part.x, part.y, p.c);
    }
    warp_merge_state<0>(m, s, unused, p.c, 0.0f);
    const int64_t r = p.row_list[i];
    const int32_t *tg = p.tgt + i * K;
    const float *xt = p.xt + i * K;
    float logp = 0.0f;
    if (lane < K) {
        float out;
        if (tg[lane] < 0) {
            out = nan_value();
            report(p.dev_status, GBCE_DEV_BAD_INDEX);
        } else {
            out = logp_with_targets<GBCE_MAX_K>(m, s, tg, xt, K, lane, p.c, p.T);
        }
        logp = out;
        if (p.logp_out != nullptr)
            p.logp_out[r * K + lane] = out;
        if (lane == 0 && p.loss_rows != nullptr)
            p.loss_rows[r] = -out;
    }
    if (lane == 0 && (p.state_out != nullptr || p.fused)) {
        for (int k = 0; k < K; ++k) {
            bool dup = tg[k] < 0;
            for (int j = 0; j < k; ++j)
                dup |= tg[j] == tg[k];
            if (!dup)
                merge_max_sum(m, s, xt[k], 1.0f, p.c);
        }
        if (p.state_out != nullptr) {
            p.state_out[2 * r] = m;
            p.state_out[2 * r + 1] = s;
        }
        if (p.fused) {
            if (i == 0)
                p.head->alpha = shared_factor(p);
            ce_row_gradient(p, i, r, m, s, logp);
        }
    }
}

// A backward call's rows, from the forward's log-probs and row states.  The
// selective gradient has (M, -G / (T S)) and, for a gathered column,
//   (-g_t expm1(log p_t) - (sum of the others' g) p_t) / T.
__global__ void __launch_bounds__(128) lin_prepare_kernel(LinParams p)
{
    grid_dependency_wait();
    launch_dependents();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i == 0)
        p.head->alpha = shared_factor(p);
    if (i >= p.head->n_live)
        return;
    const int K = static_cast<int>(p.k);
    const int64_t r = p.row_list[i];
    const float M = p.saved_state[2 * r], S = p.saved_state[2 * r + 1];
    const float *lp = p.saved_logp + r * K;
    if (p.token_ce) {
        ce_row_gradient(p, i, r, M, S, lp[0]);
        return;
    }
    const float inv_t = 1.0f / p.T;
    const float *g = p.grad_out + r * K;
    const int32_t *tg = p.tgt + i * K;
    float sum = 0.0f;
    for (int k = 0; k < K; ++k)
        sum += g[k];
    p.grow[i] = make_float2(M, -(sum * inv_t) / S);
    for (int k = 0; k < K; ++k) {
        float mine = 0.0f, other = 0.0f;
        for (int j = 0; j < K; ++j) {
            if (tg[j] == tg[k])
                mine += g[j];
            else
                other += g[j];
        }
        p.dzt[i * K + k] = (-mine * expm1f(lp[k]) - other * expf(lp[k])) * inv_t;
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
#pragma unroll 4
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

cudaError_t lin_plan(const LinParams &p, cudaStream_t s)
{
    lin_plan_kernel<<<1, kPlanThreads, 0, s>>>(p);
    note_launches(1);
    return cudaGetLastError();
}

cudaError_t lin_pack(const LinParams &p, cudaStream_t s)
{
    return launch_after(p.bf16 ? lin_pack_kernel<__nv_bfloat16, 1> : lin_pack_kernel<float, 3>,
                        dim3(static_cast<unsigned>(p.rows_pad)), dim3(128), 0, s, p);
}

cudaError_t lin_pack_weight(const LinParams &p, int64_t v0, int64_t v1, cudaStream_t s)
{
    return launch_after(p.bf16 ? lin_pack_weight_kernel<__nv_bfloat16, 1>
                               : lin_pack_weight_kernel<float, 3>,
                        dim3(static_cast<unsigned>(v1 - v0)), dim3(128), 0, s, p, v0);
}

cudaError_t lin_combine(const LinParams &p, cudaStream_t s)
{
    return launch_after(lin_combine_kernel, dim3(blocks(p.rows, 4)), dim3(128), 0, s, p);
}

cudaError_t lin_prepare(const LinParams &p, cudaStream_t s)
{
    return launch_after(lin_prepare_kernel, dim3(blocks(p.rows, 128)), dim3(128), 0, s, p);
}

cudaError_t lin_finish(const LinParams &p, cudaStream_t s)
{
    return launch_after(p.bf16 ? lin_finish_kernel<__nv_bfloat16> : lin_finish_kernel<float>,
                        dim3(static_cast<unsigned>(p.rows)), dim3(128), 0, s, p);
}

}  // namespace gbce
