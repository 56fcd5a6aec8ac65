// tcgen05 / tensor-map TMA helpers for the matrix kernels, beside the
// mbarrier helpers of gbce_device.cuh.  CTAS = 1: a CTA works on its own tile.
// CTAS = 2: the two CTAs of a cluster (a pair) work on one tile, each holding
// half of A's rows, half of B's and half of D's.
#pragma once

#include <cuda.h>

#include "gbce_device.cuh"

namespace gbce {

// ------------------------------------------------------------- tensor maps

// Box of a 3-D tensor (innermost coordinate first) into this CTA's shared
// memory; the bytes are counted on `bar`, a shared::cluster address that, in
// a pair, may lie in the other CTA.
template <int CTAS>
__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int32_t x, int32_t y,
                                            int32_t z, uint32_t bar)
{
    if constexpr (CTAS == 1) {
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
            "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
        return;
    }
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// True in one lane of a converged warp, always the same one: the commits of
// tcgen05 count the products that their own thread issued.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// 32-byte store: a whole sector per thread.  Rows of a tile lie far apart, one
// thread each, so a warp's store costs a cycle per row whatever its width.
__device__ __forceinline__ void st_v8(void *p, const uint32_t (&w)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

__device__ __forceinline__ void st_v8(float *p, const float *v)
{
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w[i] = __float_as_uint(v[i]);
    st_v8(static_cast<void *>(p), w);
}

// ------------------------------------------------------------ cluster sync

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
                 ::: "memory");
}

// Arrive on an mbarrier at a shared::cluster address.  What it tells the other
// CTA is that TMEM has been read (ordered by the tcgen05 fence before it), no
// memory that this CTA wrote: at cluster scope the release would wait for the
// thread's global stores, which are a tile's outputs.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// ------------------------------------------------------------------- TMEM

// One whole warp of the CTA (of each of a pair's) calls these.
template <int CTAS>
__device__ __forceinline__ void tmem_alloc(uint32_t *slot, uint32_t columns)
{
    if constexpr (CTAS == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(slot)),
                     "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(slot)),
                     "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
}

template <int CTAS>
__device__ __forceinline__ void tmem_free(uint32_t taddr, uint32_t columns)
{
    if constexpr (CTAS == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr),
                     "r"(columns)
                     : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr),
                     "r"(columns)
                     : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 lanes x 16 columns of fp32: thread l gets columns [col, col + 16) of its
// warp's lane l, added to what v holds (`fresh`: instead of it).
__device__ __forceinline__ void tmem_add16(uint32_t taddr, float *v, bool fresh)
{
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        const float2 x = make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1]));
        const float2 y = fresh ? x : fadd2(make_float2(v[i], v[i + 1]), x);
        v[i] = y.x;
        v[i + 1] = y.y;
    }
}

// -------------------------------------------------------------------- MMA

// Shared-memory matrix descriptor, 128-byte swizzle.  Offsets in bytes.
// K-major (rows of 64 bf16 along k): groups of 8 rows are `sbo` apart.
// MN-major (rows of 64 bf16 along m or n): 64-wide chunks are `lbo` apart,
// groups of 8 k-rows `sbo` apart.
__device__ __forceinline__ uint64_t mma_desc(uint32_t addr, uint32_t lbo, uint32_t sbo)
{
    return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) |
           (static_cast<uint64_t>((lbo >> 4) & 0x3fffu) << 16) |
           (static_cast<uint64_t>((sbo >> 4) & 0x3fffu) << 32) | (uint64_t{1} << 46) |
           (uint64_t{2} << 61);
}

// Instruction descriptor of kind::f16 with bf16 operands and fp32 sums.
__host__ __device__ constexpr uint32_t mma_idesc(uint32_t m, uint32_t n, bool a_mn, bool b_mn)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(a_mn) << 15) |
           (static_cast<uint32_t>(b_mn) << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

template <int CTAS>
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         bool accumulate)
{
    if constexpr (CTAS == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
            : "memory");
}

// One arrival on `bar` (in a pair: on the barrier at the same offset in both
// CTAs) once every MMA issued so far by this thread is done.
template <int CTAS>
__device__ __forceinline__ void mma_commit(uint64_t *bar)
{
    if constexpr (CTAS == 2)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
            " [%0], %1;" ::"r"(smem_addr(bar)),
            "h"(static_cast<uint16_t>(3))
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                     ::"r"(smem_addr(bar))
                     : "memory");
}

}  // namespace gbce
