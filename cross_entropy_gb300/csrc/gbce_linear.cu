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

// Packed hidden states and targets of the live rows, one CTA per packed row;
// the rows up to the next multiple of kLinRowPad are zeros.
template <typename T>
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
    const T *src = static_cast<const T *>(p.hidden) + r * p.hidden_stride;
    T *dst = static_cast<T *>(p.hpack) + i * p.dim;
    for (int64_t d = threadIdx.x; d < p.dim; d += blockDim.x)
        dst[d] = in ? src[d] : T(0.0f);
    const int K = static_cast<int>(p.k);
    for (int k = threadIdx.x; k < K; k += blockDim.x) {
        const int64_t t = in ? p.targets[r * K + k] : -1;
        p.tgt[i * K + k] = t >= 0 && t < p.vocab ? static_cast<int32_t>(t) : -1;
    }
}

// ------------------------------------------------------------ simple products

constexpr int kSgT = 64, kSgK = 16;

// One 64 x 64 tile of A . B over k: 256 threads, 4 x 4 values each, every
// product and sum in fp32.  A(m, k) = a[m am + k ak], B(n, k) = b[n bn + k bk].
template <typename TA, typename TB>
__device__ void simple_tile(const TA *a, int64_t am, int64_t ak, int64_t m0, int64_t mlim,
                            const TB *b, int64_t bn, int64_t bk, int64_t n0, int64_t nlim,
                            int64_t klim, float (&acc)[4][4], float *sm)
{
    float *sa = sm, *sb = sm + kSgK * (kSgT + 1);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[i][j] = 0.0f;
    for (int64_t k0 = 0; k0 < klim; k0 += kSgK) {
        for (int e = threadIdx.x; e < kSgT * kSgK; e += 256) {
            const int row = ak == 1 ? e / kSgK : e % kSgT, kk = ak == 1 ? e % kSgK : e / kSgT;
            const bool in = m0 + row < mlim && k0 + kk < klim;
            sa[kk * (kSgT + 1) + row] = in ? static_cast<float>(a[(m0 + row) * am + (k0 + kk) * ak])
                                           : 0.0f;
        }
        for (int e = threadIdx.x; e < kSgT * kSgK; e += 256) {
            const int row = bk == 1 ? e / kSgK : e % kSgT, kk = bk == 1 ? e % kSgK : e / kSgT;
            const bool in = n0 + row < nlim && k0 + kk < klim;
            sb[kk * (kSgT + 1) + row] = in ? static_cast<float>(b[(n0 + row) * bn + (k0 + kk) * bk])
                                           : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < kSgK; ++kk) {
            float x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = sa[kk * (kSgT + 1) + ty * 4 + i];
                y[i] = sb[kk * (kSgT + 1) + tx * 4 + i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
        }
        __syncthreads();
    }
}

constexpr int kSgSmem = kSgT * (kSgT + 1);  // floats; holds the operands, then the tile

// Logits of a 64 x 64 tile into shared memory.
template <typename T>
__device__ void simple_logits(const LinParams &p, int64_t i0, int64_t v0, int32_t live, float *sm)
{
    float acc[4][4];
    simple_tile(static_cast<const T *>(p.hpack), p.dim, 1, i0, live,
                static_cast<const T *>(p.weight), p.weight_stride, 1, v0, p.vocab, p.dim, acc, sm);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            sm[(ty * 4 + i) * (kSgT + 1) + tx * 4 + j] = acc[i][j];
    __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(256) lin_stats_simple(LinParams p)
{
    __shared__ float sm[kSgSmem];
    const int32_t live = p.head->n_live;
    const int64_t i0 = static_cast<int64_t>(blockIdx.y) * kSgT;
    if (i0 >= live)
        return;
    const int K = static_cast<int>(p.k);
    float m = kNegInf, s = 0.0f;
    const int64_t i = i0 + threadIdx.x;
    for (int64_t v0 = static_cast<int64_t>(blockIdx.x) * kLinTileV;
         v0 < min(p.vocab, (static_cast<int64_t>(blockIdx.x) + 1) * kLinTileV); v0 += kSgT) {
        simple_logits<T>(p, i0, v0, live, sm);
        if (threadIdx.x < kSgT && i < live) {
            float *row = sm + threadIdx.x * (kSgT + 1);
            const int n = static_cast<int>(min(static_cast<int64_t>(kSgT), p.vocab - v0));
            // a column gathered twice is read before the first of them masks it
            for (int k = 0; k < K; ++k) {
                const int64_t j = p.tgt[i * K + k] - v0;
                if (j >= 0 && j < n)
                    p.xt[i * K + k] = row[j];
            }
            for (int k = 0; k < K; ++k) {
                const int64_t j = p.tgt[i * K + k] - v0;
                if (j >= 0 && j < n)
                    row[j] = kNegInf;
            }
            float tm = kNegInf;
            for (int j = 0; j < n; ++j)
                tm = fmaxf(tm, row[j]);
            const float ref = tm == kNegInf ? 0.0f : tm;
            float ts = 0.0f;
            for (int j = 0; j < n; ++j)
                ts += ex2((row[j] - ref) * p.c);
            // a tile of NaNs has no max, and keeps its NaN sum
            merge_max_sum(m, s, ts == ts ? tm : ref, ts, p.c);
        }
        __syncthreads();
    }
    if (threadIdx.x < kSgT && i < live)
        p.partials[i * p.tiles + blockIdx.x] = make_float2(m, s);
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
    if (lane < K) {
        float out;
        if (tg[lane] < 0) {
            out = nan_value();
            report(p.dev_status, GBCE_DEV_BAD_INDEX);
        } else {
            out = logp_with_targets<GBCE_MAX_K>(m, s, tg, xt, K, lane, p.c, p.T);
        }
        if (p.logp_out != nullptr)
            p.logp_out[r * K + lane] = out;
        if (lane == 0 && p.loss_rows != nullptr)
            p.loss_rows[r] = -out;
    }
    if (lane == 0 && p.state_out != nullptr) {
        for (int k = 0; k < K; ++k) {
            bool dup = tg[k] < 0;
            for (int j = 0; j < k; ++j)
                dup |= tg[j] == tg[k];
            if (!dup)
                merge_max_sum(m, s, xt[k], 1.0f, p.c);
        }
        p.state_out[2 * r] = m;
        p.state_out[2 * r + 1] = s;
    }
}

// What the gradient of a row takes besides its logits: (M, coef / S), and
// the dz of its gathered columns,
//   -u_t expm1(log p_t) - (sum of the others' u) p_t,   u = upstream / T,
// in which 1 - p_t keeps its value when p_t rounds to 1.  The factor that
// all rows share (a summed or averaged loss's) stays out of dz: it joins at
// the end, in fp32, so that it is not rounded with each dz.
__global__ void __launch_bounds__(128) lin_prepare_kernel(LinParams p)
{
    grid_dependency_wait();
    launch_dependents();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    const float inv_t = 1.0f / p.T;
    if (i == 0) {
        double a = 1.0;
        if (p.token_ce && p.reduction != 0) {
            a = static_cast<double>(p.grad_out[0]) / static_cast<double>(p.T);
            if (p.reduction == 2) {
                const int64_t n = p.n_items != nullptr ? *p.n_items : p.head->n_items;
                a = n > 0 ? a / static_cast<double>(n) : 0.0;
            }
        }
        p.head->alpha = static_cast<float>(a);
    }
    if (i >= p.head->n_live)
        return;
    const int K = static_cast<int>(p.k);
    const int64_t r = p.row_list[i];
    const float M = p.saved_state[2 * r], S = p.saved_state[2 * r + 1];
    const float *lp = p.saved_logp + r * K;
    if (p.token_ce) {
        const float u = p.reduction == 0 ? p.grad_out[r] * inv_t : 1.0f;
        p.grow[i] = make_float2(M, u / S);
        p.dzt[i] = u * expm1f(lp[0]);
        return;
    }
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

// dz of one piece of the vocabulary [v0, v1), in the inputs' type.
template <typename T>
__global__ void __launch_bounds__(256) lin_dz_simple(LinParams p, int64_t v0, int64_t v1)
{
    __shared__ float sm[kSgSmem];
    const int32_t live = p.head->n_live;
    const int64_t i0 = static_cast<int64_t>(blockIdx.y) * kSgT;
    if (i0 >= live)
        return;
    const int64_t c0 = v0 + static_cast<int64_t>(blockIdx.x) * kSgT;
    simple_logits<T>(p, i0, c0, live, sm);
    T *dz = static_cast<T *>(p.dz);
    for (int e = threadIdx.x; e < kSgT * kSgT; e += 256) {
        const int64_t i = i0 + e / kSgT, v = c0 + e % kSgT;
        if (i < live && v < v1) {
            const float2 g = p.grow[i];
            dz[i * p.piece + v - v0] = T(g.y * ex2((sm[e / kSgT * (kSgT + 1) + e % kSgT] - g.x) * p.c));
        }
    }
    __syncthreads();
    const int64_t i = i0 + threadIdx.x;
    if (threadIdx.x < kSgT && i < live)
        for (int k = 0; k < p.k; ++k) {
            const int64_t v = p.tgt[i * p.k + k];
            if (v >= c0 && v < min(v1, c0 + kSgT))
                dz[i * p.piece + v - v0] = T(p.dzt[i * p.k + k]);
        }
}

// dh (+)= dz . weight over one piece.
template <typename T>
__global__ void __launch_bounds__(256) lin_dh_simple(LinParams p, int64_t v0, int64_t v1)
{
    __shared__ float sm[kSgSmem];
    const int32_t live = p.head->n_live;
    const int64_t i0 = static_cast<int64_t>(blockIdx.y) * kSgT, d0 = static_cast<int64_t>(blockIdx.x) * kSgT;
    if (i0 >= live)
        return;
    float acc[4][4];
    simple_tile(static_cast<const T *>(p.dz), p.piece, 1, i0, live,
                static_cast<const T *>(p.weight) + v0 * p.weight_stride, 1, p.weight_stride, d0,
                p.dim, v1 - v0, acc, sm);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int a = 0; a < 4; ++a)
        for (int b = 0; b < 4; ++b) {
            const int64_t i = i0 + ty * 4 + a, d = d0 + tx * 4 + b;
            if (i < live && d < p.dim) {
                float *o = p.dh + i * p.dim + d;
                *o = v0 == 0 ? acc[a][b] : *o + acc[a][b];
            }
        }
}

// dweight rows of one piece, (+)= alpha dz^T . hidden.
template <typename T>
__global__ void __launch_bounds__(256) lin_dw_simple(LinParams p, int64_t v0, int64_t v1)
{
    __shared__ float sm[kSgSmem];
    const int32_t live = p.head->n_live;
    const float alpha = p.head->alpha;
    const int64_t c0 = static_cast<int64_t>(blockIdx.y) * kSgT, d0 = static_cast<int64_t>(blockIdx.x) * kSgT;
    float acc[4][4];
    simple_tile(static_cast<const T *>(p.dz), 1, p.piece, c0, v1 - v0,
                static_cast<const T *>(p.hpack), 1, p.dim, d0, p.dim, live, acc, sm);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int a = 0; a < 4; ++a)
        for (int b = 0; b < 4; ++b) {
            const int64_t v = v0 + c0 + ty * 4 + a, d = d0 + tx * 4 + b;
            if (v < v1 && d < p.dim) {
                T *o = static_cast<T *>(p.dweight) + v * p.dweight_stride + d;
                const float x = alpha * acc[a][b];
                *o = T(p.accumulate ? static_cast<float>(*o) + x : x);
            }
        }
}

// dhidden by original row: alpha times the sums, zeros for rows left out,
// NaN for rows with a target out of range.
template <typename T>
__global__ void __launch_bounds__(128) lin_finish_kernel(LinParams p)
{
    grid_dependency_wait();
    launch_dependents();
    const int64_t r = blockIdx.x;
    const int32_t i = p.row_map[r];
    const float alpha = p.head->alpha;
    T *out = static_cast<T *>(p.dhidden) + r * p.dhidden_stride;
    for (int64_t d = threadIdx.x; d < p.dim; d += blockDim.x) {
        const float x = i >= 0 ? alpha * p.dh[i * p.dim + d]
                               : (i == kLinRowBad ? nan_value() : 0.0f);
        out[d] = T(x);
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
    return launch_after(p.bf16 ? lin_pack_kernel<__nv_bfloat16> : lin_pack_kernel<float>,
                        dim3(static_cast<unsigned>(p.rows_pad)), dim3(128), 0, s, p);
}

cudaError_t lin_stats(const LinParams &p, cudaStream_t s)
{
    const dim3 grid(static_cast<unsigned>(p.tiles), blocks(p.rows, kSgT));
    if (p.bf16)
        lin_stats_simple<__nv_bfloat16><<<grid, 256, 0, s>>>(p);
    else
        lin_stats_simple<float><<<grid, 256, 0, s>>>(p);
    note_launches(1);
    return cudaGetLastError();
}

cudaError_t lin_combine(const LinParams &p, cudaStream_t s)
{
    return launch_after(lin_combine_kernel, dim3(blocks(p.rows, 4)), dim3(128), 0, s, p);
}

cudaError_t lin_prepare(const LinParams &p, cudaStream_t s)
{
    return launch_after(lin_prepare_kernel, dim3(blocks(p.rows, 128)), dim3(128), 0, s, p);
}

template <typename T>
static cudaError_t grads(const LinParams &p, cudaStream_t s)
{
    for (int64_t v0 = 0; v0 < p.vocab; v0 += p.piece) {
        const int64_t v1 = v0 + p.piece < p.vocab ? v0 + p.piece : p.vocab;
        lin_dz_simple<T><<<dim3(blocks(v1 - v0, kSgT), blocks(p.rows, kSgT)), 256, 0, s>>>(p, v0, v1);
        note_launches(1);
        if (p.dhidden != nullptr) {
            lin_dh_simple<T><<<dim3(blocks(p.dim, kSgT), blocks(p.rows, kSgT)), 256, 0, s>>>(p, v0, v1);
            note_launches(1);
        }
        if (p.dweight != nullptr) {
            lin_dw_simple<T><<<dim3(blocks(p.dim, kSgT), blocks(v1 - v0, kSgT)), 256, 0, s>>>(p, v0, v1);
            note_launches(1);
        }
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess)
            return e;
    }
    if (p.dhidden == nullptr)
        return cudaSuccess;
    return launch_after(lin_finish_kernel<T>, dim3(static_cast<unsigned>(p.rows)), dim3(128), 0, s, p);
}

cudaError_t lin_grads(const LinParams &p, cudaStream_t s)
{
    return p.bf16 ? grads<__nv_bfloat16>(p, s) : grads<float>(p, s);
}

}  // namespace gbce
