// Reading rows of hidden states and weights, of any alignment, eight elements
// at a time.
#pragma once

#include "gbce_device.cuh"

namespace gbce {

// Eight elements of a row from any element on, as fp32.  `aligned`: from 16
// bytes.  Otherwise bf16 goes by whole 4-byte words, shifted where the row
// starts between two (in which case the word before the first element and the
// one after the last are read too: read_eight keeps off the row's ends).
__device__ __forceinline__ void load_eight(const __nv_bfloat16 *p, bool aligned, float (&x)[8])
{
    uint32_t w[4];
    if (aligned) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
        const uint32_t between = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 2u);
        const uint32_t *q = reinterpret_cast<const uint32_t *>(reinterpret_cast<uintptr_t>(p) - between);
        uint32_t u[5];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            u[i] = __ldg(q + i);
        u[4] = between != 0 ? __ldg(q + 4) : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = __funnelshift_r(u[i], u[i + 1], between * 8);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = bf16x2_to_float2(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ void load_eight(const float *p, bool aligned, float (&x)[8])
{
    if (aligned) {
        const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = __ldg(p + i);
    }
}

// Elements [d, d + 8) of a row of dim, zeros past its end.
template <typename T>
__device__ __forceinline__ void read_eight(const T *row, int64_t d, int64_t dim, float (&x)[8])
{
    const bool aligned = reinterpret_cast<uintptr_t>(row) % 16 == 0;
    if (d + 8 <= dim && (aligned || (d > 0 && d + 8 < dim))) {
        load_eight(row + d, aligned, x);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = d + i < dim ? static_cast<float>(row[d + i]) : 0.0f;
    }
}

__device__ __forceinline__ void as_floats(const uint4 &v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = bf16x2_to_float2(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// Product of two rows by a warp, in fp32 throughout: 256 running sums, each
// of dim / 256 terms, joined by a tree.  Every lane has the result, whose bits
// do not depend on the rows' alignment.  A warp makes few of these, so what
// counts is the wait for memory: whole rows on 16 bytes go 64 bf16 (or 32 fp32)
// of each at a time.
template <typename T>
__device__ __forceinline__ float row_dot(const T *a, const T *b, int64_t dim)
{
    float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    int64_t d = 8 * static_cast<int64_t>(threadIdx.x & 31);
    if ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) % 16 == 0) {
        constexpr int kParts = sizeof(T) / 2, kAhead = 8 / kParts;
        for (; d + 8 <= dim; d += 256 * kAhead) {
            uint4 x[kAhead][kParts], y[kAhead][kParts];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const bool in = d + 256 * u + 8 <= dim;
#pragma unroll
                for (int i = 0; i < kParts; ++i) {
                    x[u][i] = y[u][i] = make_uint4(0, 0, 0, 0);
                    if (in) {
                        x[u][i] = __ldg(reinterpret_cast<const uint4 *>(a + d + 256 * u) + i);
                        y[u][i] = __ldg(reinterpret_cast<const uint4 *>(b + d + 256 * u) + i);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                float p[8], q[8];
                if constexpr (kParts == 1) {
                    as_floats(x[u][0], p);
                    as_floats(y[u][0], q);
                } else {
#pragma unroll
                    for (int i = 0; i < kParts; ++i) {
                        const uint4 &v = x[u][i], &w = y[u][i];
                        p[4 * i] = __uint_as_float(v.x), p[4 * i + 1] = __uint_as_float(v.y);
                        p[4 * i + 2] = __uint_as_float(v.z), p[4 * i + 3] = __uint_as_float(v.w);
                        q[4 * i] = __uint_as_float(w.x), q[4 * i + 1] = __uint_as_float(w.y);
                        q[4 * i + 2] = __uint_as_float(w.z), q[4 * i + 3] = __uint_as_float(w.w);
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    acc[i] = fmaf(p[i], q[i], acc[i]);
            }
        }
        // the one part that the rows' end cuts, if it is this lane's
        d = dim % 8 != 0 && (dim & ~int64_t{7}) % 256 == 8 * static_cast<int64_t>(threadIdx.x & 31) ? dim & ~int64_t{7} : dim;
    }
#pragma unroll 2
    for (; d < dim; d += 256) {
        float x[8], y[8];
        read_eight(a, d, dim, x);
        read_eight(b, d, dim, y);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc[i] = fmaf(x[i], y[i], acc[i]);
    }
    return warp_sum(((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7])));
}

}  // namespace gbce
