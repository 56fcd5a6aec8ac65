// Rows of a [vocab, dim] table by token, and the gradient of that lookup.
//
//   out[r]    = scale * table[token[r]]               (0 where the token is ignored)
//   dtable[v] (+)= scale * sum_{r : token[r] = v} grad[r]
//
// Both are copies of rows: bound by memory.
#include <cmath>
#include <cstdint>

#include "gbce_kernels.cuh"

namespace gbce {

namespace {

// Columns [d0, d0 + 16 bytes) of a row as fp32.
template <typename T>
__device__ __forceinline__ float scaled(T x, float scale)
{
    return static_cast<float>(x) * scale;
}

}  // namespace

template <typename T>
__global__ void __launch_bounds__(128)
    embedding_lookup_kernel(const T *table, int64_t table_stride, int64_t vocab, int64_t dim,
                            const int64_t *tokens, int64_t ignore_index, float scale, T *out,
                            int64_t out_stride, int32_t *dev_status)
{
    const int64_t r = blockIdx.x;
    const int64_t t = tokens[r];
    T *dst = out + r * out_stride;
    const bool skip = t == ignore_index;
    if (skip || t < 0 || t >= vocab) {
        if (!skip && threadIdx.x == 0)
            report(dev_status, GBCE_DEV_BAD_INDEX);
        const T fill = T(skip ? 0.0f : __int_as_float(0x7fc00000));
        for (int64_t d = threadIdx.x; d < dim; d += blockDim.x)
            dst[d] = fill;
        return;
    }
    const T *src = table + t * table_stride;
    for (int64_t d = threadIdx.x; d < dim; d += blockDim.x)
        dst[d] = T(scaled(src[d], scale));
}

// One CTA per table row: its tokens in order, 128 columns at a time.
template <typename T>
__global__ void __launch_bounds__(128)
    embedding_grad_kernel(const T *grad, int64_t grad_stride, int64_t rows, int64_t vocab,
                          int64_t dim, const int64_t *tokens, int64_t ignore_index, float scale,
                          T *dtable, int64_t dtable_stride, int accumulate, int32_t *dev_status)
{
    __shared__ int32_t s_row[128];
    __shared__ int32_t s_n[4];
    const int64_t v = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (v == 0)
        for (int64_t r = threadIdx.x; r < rows; r += blockDim.x)
            if (tokens[r] != ignore_index && (tokens[r] < 0 || tokens[r] >= vocab))
                report(dev_status, GBCE_DEV_BAD_INDEX);
    for (int64_t d0 = 0; d0 < dim; d0 += blockDim.x) {
        const int64_t d = d0 + threadIdx.x;
        float sum = 0.0f;
        bool any = false;
        for (int64_t r0 = 0; r0 < rows; r0 += 128) {
            const int64_t r = r0 + threadIdx.x;
            const bool hit = r < rows && tokens[r] == v && v != ignore_index;
            const unsigned b = __ballot_sync(0xffffffffu, hit);
            if (lane == 0)
                s_n[warp] = __popc(b);
            __syncthreads();
            int before = 0;
            for (int w = 0; w < warp; ++w)
                before += s_n[w];
            if (hit)
                s_row[before + __popc(b & ((1u << lane) - 1u))] = static_cast<int32_t>(r - r0);
            const int n = s_n[0] + s_n[1] + s_n[2] + s_n[3];
            __syncthreads();
            if (d < dim)
                for (int j = 0; j < n; ++j)
                    sum += static_cast<float>(grad[(r0 + s_row[j]) * grad_stride + d]);
            any |= n > 0;
            __syncthreads();
        }
        if (d < dim) {
            T *o = dtable + v * dtable_stride + d;
            if (!accumulate)
                *o = T(sum * scale);
            else if (any)
                *o = T(fmaf(sum, scale, static_cast<float>(*o)));
        }
    }
}

}  // namespace gbce

namespace {

size_t elem_size(gbce_dtype dt) { return dt == GBCE_BF16 ? 2 : 4; }

constexpr int64_t kMaxVocab = INT32_MAX - 64;

gbce_status check_table(const void *p, int64_t n, int64_t stride, int64_t dim, gbce_dtype dt)
{
    if (p == nullptr || stride < dim || stride > (INT64_MAX / 16) / (n > 0 ? n : 1))
        return GBCE_EINVAL;
    return reinterpret_cast<uintptr_t>(p) % elem_size(dt) == 0 ? GBCE_OK : GBCE_EDTYPE;
}

bool overlap(const void *a, int64_t an, int64_t as, const void *b, int64_t bn, int64_t bs,
             int64_t dim, gbce_dtype dt)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    const size_t xb = static_cast<size_t>((an - 1) * as + dim) * elem_size(dt);
    const size_t yb = static_cast<size_t>((bn - 1) * bs + dim) * elem_size(dt);
    return x < y + yb && y < x + xb;
}

gbce_status check_sizes(gbce_dtype dtype, int64_t rows, int64_t vocab, int64_t dim, float scale)
{
    if (dtype != GBCE_F32 && dtype != GBCE_BF16)
        return GBCE_EDTYPE;
    if (rows < 0 || rows > INT32_MAX / 2 || vocab < 1 || vocab > kMaxVocab || dim < 1 ||
        dim > (int64_t{1} << 20) || !std::isfinite(scale))
        return GBCE_EINVAL;
    return GBCE_OK;
}

template <typename T>
cudaError_t lookup(const void *table, int64_t ts, int64_t vocab, int64_t dim, const int64_t *tokens,
                   int64_t rows, int64_t ignore_index, float scale, void *out, int64_t os,
                   int32_t *dev_status, cudaStream_t s)
{
    gbce::embedding_lookup_kernel<T><<<static_cast<unsigned>(rows), 128, 0, s>>>(
        static_cast<const T *>(table), ts, vocab, dim, tokens, ignore_index, scale,
        static_cast<T *>(out), os, dev_status);
    gbce::note_launches(1);
    return cudaGetLastError();
}

template <typename T>
cudaError_t lookup_bwd(const void *grad, int64_t gs, int64_t rows, int64_t vocab, int64_t dim,
                       const int64_t *tokens, int64_t ignore_index, float scale, void *dtable,
                       int64_t ds, int accumulate, int32_t *dev_status, cudaStream_t s)
{
    gbce::embedding_grad_kernel<T><<<static_cast<unsigned>(vocab), 128, 0, s>>>(
        static_cast<const T *>(grad), gs, rows, vocab, dim, tokens, ignore_index, scale,
        static_cast<T *>(dtable), ds, accumulate, dev_status);
    gbce::note_launches(1);
    return cudaGetLastError();
}

}  // namespace

extern "C" {

size_t gbce_embedding_workspace_size(int64_t rows, int64_t vocab, int64_t dim)
{
    return rows > 0 && vocab > 0 && dim > 0 ? 256 : 0;
}

gbce_status embedding_lookup(const void *table, int64_t table_row_stride, gbce_dtype dtype,
                             int64_t vocab, int64_t dim, const int64_t *tokens, int64_t rows,
                             int64_t ignore_index, float scale, void *out, int64_t out_row_stride,
                             int32_t *dev_status, void *stream)
{
    gbce_status st = check_sizes(dtype, rows, vocab, dim, scale);
    if (st != GBCE_OK || rows == 0)
        return st;
    if ((st = check_table(table, vocab, table_row_stride, dim, dtype)) != GBCE_OK ||
        (st = check_table(out, rows, out_row_stride, dim, dtype)) != GBCE_OK)
        return st;
    if (tokens == nullptr ||
        overlap(table, vocab, table_row_stride, out, rows, out_row_stride, dim, dtype))
        return GBCE_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e =
        dtype == GBCE_BF16
            ? lookup<__nv_bfloat16>(table, table_row_stride, vocab, dim, tokens, rows, ignore_index,
                                    scale, out, out_row_stride, dev_status, s)
            : lookup<float>(table, table_row_stride, vocab, dim, tokens, rows, ignore_index, scale,
                            out, out_row_stride, dev_status, s);
    return e == cudaSuccess ? GBCE_OK : GBCE_ECUDA;
}

gbce_status embedding_lookup_bwd(const void *grad_out, int64_t grad_row_stride, gbce_dtype dtype,
                                 int64_t rows, int64_t dim, const int64_t *tokens, int64_t vocab,
                                 int64_t ignore_index, float scale, void *dtable,
                                 int64_t dtable_row_stride, int accumulate, void *workspace,
                                 size_t workspace_bytes, int32_t *dev_status, void *stream)
{
    gbce_status st = check_sizes(dtype, rows, vocab, dim, scale);
    if (st != GBCE_OK)
        return st;
    if ((st = check_table(dtable, vocab, dtable_row_stride, dim, dtype)) != GBCE_OK)
        return st;
    if (rows > 0) {
        if ((st = check_table(grad_out, rows, grad_row_stride, dim, dtype)) != GBCE_OK)
            return st;
        if (tokens == nullptr ||
            overlap(dtable, vocab, dtable_row_stride, grad_out, rows, grad_row_stride, dim, dtype))
            return GBCE_EINVAL;
        if (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 16 != 0 ||
            workspace_bytes < gbce_embedding_workspace_size(rows, vocab, dim))
            return GBCE_EWORKSPACE;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e =
        dtype == GBCE_BF16
            ? lookup_bwd<__nv_bfloat16>(grad_out, grad_row_stride, rows, vocab, dim, tokens,
                                        ignore_index, scale, dtable, dtable_row_stride, accumulate,
                                        dev_status, s)
            : lookup_bwd<float>(grad_out, grad_row_stride, rows, vocab, dim, tokens, ignore_index,
                                scale, dtable, dtable_row_stride, accumulate, dev_status, s);
    return e == cudaSuccess ? GBCE_OK : GBCE_ECUDA;
}

}  // extern "C"
