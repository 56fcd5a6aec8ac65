// The matrix products of the calls that start from hidden states, on the
// tensor cores: one kernel, four uses.
//
//   stats  logits = hidden . weight^T    -> (max, sum) per row and 256 columns
//   dz     the same logits again         -> dz, in memory for one piece
//   dh     dz . weight                   -> dhidden sums (fp32)
//   dw     dz^T . hidden                 -> dweight rows of the piece
//
// A pair of CTAs works on a 256 x 256 tile: TMA brings 64-deep slices of both
// operands into a six-stage ring (32 KB a stage and CTA), one thread of the
// pair issues the MMAs (M = 256 across the pair), and the sums lie in TMEM,
// two tiles' worth (2 x 256 columns), so that four warps turn one tile into
// outputs while the next is multiplied.  Persistent: one pair per two SMs.
//
// Operands are read in the layout they have: hidden, weight and dz lie with
// the product's depth innermost for stats and dz (and dz for dh), and with it
// outermost for dh's weight and both operands of dw; the matrix descriptors
// take either, so that nothing is ever transposed in memory.
//
// fp32 inputs come as three bf16 planes, x = hi + mid + lo with 8 more bits
// in each; six of the nine products (all above 2^-24 of x y) are summed,
// smallest first, so that the large ones meet a sum that is still small.
#include <cuda.h>

#include "gbce_kernels.cuh"
#include "gbce_linear.h"
#include "gbce_umma.cuh"

namespace gbce {

namespace {

constexpr int kRing = 6;
constexpr int kTile = 256;           // rows and columns of a pair's tile
constexpr int kDepth = 64;           // depth of a stage: 128 bytes of bf16
constexpr uint32_t kHalfBytes = 128 * kDepth * 2;  // a CTA's half of one operand
constexpr uint32_t kStageBytes = 2 * kHalfBytes;
constexpr int kMmaThreads = 192;     // TMA warp, MMA warp, four epilogue warps
constexpr uint32_t kTmemCols = 512;

enum LinMode : int { kLinStats, kLinDz, kLinDh, kLinDw };

struct MmaArgs {
    const LinHeader *head;
    int32_t *dev_status;
    int32_t pairs;         // plane products: 1, or 6 for fp32 inputs
    int32_t depth;         // elements of the depth (dw: the live rows)
    int32_t tiles_m;       // dw: tiles of the piece; else from the live rows
    int32_t tiles_n;
    int32_t splits;        // dh: parts of the depth
    int32_t b_row0;        // stats, dz, dh: the piece's first row in the weight's map
    int64_t v0, vocab;     // first column of the piece; end of the vocabulary
    float c;
    int32_t k;
    const int32_t *tgt;
    float *xt;
    float2 *partials;
    int64_t partial_tiles;
    const float2 *grow;
    const float *dzt;
    __nv_bfloat16 *dz;
    int64_t piece, dz_plane;
    int32_t planes;
    float *dh;
    int64_t dim, dh_pitch, dh_split;
    void *dweight;
    int64_t dweight_stride;
    int32_t first, accumulate, bf16, vec;
};

struct MmaShared {
    uint64_t full[kRing], empty[kRing], acc_full[2], acc_empty[2];
    uint32_t tmem;
    int32_t failed;
};

constexpr uint32_t kSmemBytes = kRing * kStageBytes + sizeof(MmaShared) + 1024;

struct TileId {
    int32_t m, n, split;
};

// Tiles in an order that keeps both operands in L2 while they are needed.
// stats, dz: all row tiles (hidden stays in L2) before the next columns, so
// that the table is read once.  dh, dw: bands of 8 tiles high, so that the
// pairs at work cover a block that is about square.
template <int MODE>
__device__ __forceinline__ TileId tile_of(int64_t t, int32_t tm, int32_t tn)
{
    TileId r;
    if (MODE == kLinStats || MODE == kLinDz) {
        r.m = static_cast<int32_t>(t % tm);
        r.n = static_cast<int32_t>(t / tm);
        r.split = 0;
        return r;
    }
    const int64_t per = static_cast<int64_t>(tm) * tn;
    r.split = static_cast<int32_t>(t / per);
    const int32_t u = static_cast<int32_t>(t % per);
    const int32_t band = u / (8 * tn), in = u % (8 * tn);
    const int32_t high = min(8, tm - band * 8);
    r.m = band * 8 + in % high;
    r.n = in / high;
    return r;
}

// Plane indices of product q of six, smallest first.
__device__ __forceinline__ int plane_a(int pairs, int q) { return pairs == 1 ? 0 : (0x201100 >> (4 * (5 - q))) & 15; }
__device__ __forceinline__ int plane_b(int pairs, int q) { return pairs == 1 ? 0 : (0x021010 >> (4 * (5 - q))) & 15; }

__device__ __forceinline__ bool wait_or_fail(uint64_t *bar, uint32_t parity, MmaShared *sh,
                                             int32_t *dev_status)
{
    if (mbar_wait_cluster(bar, parity))
        return true;
    *reinterpret_cast<volatile int32_t *>(&sh->failed) = 1;
    report(dev_status, GBCE_DEV_TIMEOUT);
    return false;
}

// ------------------------------------------------------------- epilogues
// One thread has one row of the tile; `col` is its first column in the tile.

struct RowStats {
    float m = kNegInf, s = 0.0f;

    __device__ __forceinline__ void add(const float (&v)[32], float c)
    {
        float a = kNegInf, b = kNegInf;
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
            a = fmax3(a, v[j], v[j + 1]);
            b = fmax3(b, v[j + 2], v[j + 3]);
        }
        const float top = fmax3(a, b, m);
        const float ref = top == kNegInf ? 0.0f : top;
        float2 s0 = make_float2(0.0f, 0.0f), s1 = s0;
        const float2 r2 = make_float2(-ref, -ref), c2 = make_float2(c, c);
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
            const float2 x = fmul2(fadd2(make_float2(v[j], v[j + 1]), r2), c2);
            const float2 y = fmul2(fadd2(make_float2(v[j + 2], v[j + 3]), r2), c2);
            s0 = fadd2(s0, make_float2(ex2(x.x), ex2(x.y)));
            s1 = fadd2(s1, make_float2(ex2(y.x), ex2(y.y)));
        }
        const float sum = (s0.x + s0.y) + (s1.x + s1.y);
        s = fmaf(s, ex2((m - ref) * c), sum);
        m = top;
    }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    return float2_to_bf16x2(make_float2(lo, hi));
}

}  // namespace

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMmaThreads, 1)
    lin_mma_kernel(const __grid_constant__ CUtensorMap map_a,
                   const __grid_constant__ CUtensorMap map_b, const __grid_constant__ MmaArgs q)
{
    extern __shared__ uint8_t raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t{1023});
    MmaShared *sh = reinterpret_cast<MmaShared *>(ring + kRing * kStageBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    if (threadIdx.x == 0) {
        tma_prefetch_map(&map_a);
        tma_prefetch_map(&map_b);
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&sh->full[i], 1);
            mbar_init(&sh->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->acc_full[i], 1);
            mbar_init(&sh->acc_empty[i], 8);  // four warps of each CTA
        }
        sh->failed = 0;
        fence_barrier_init();
    }
    if (warp == 1)
        tmem_alloc_pair(&sh->tmem, kTmemCols);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before either signals them
    tc_fence_after();
    const uint32_t tmem = sh->tmem;

    grid_dependency_wait();
    launch_dependents();
    const int32_t live = q.head->n_live;
    const int32_t tm = MODE == kLinDw ? q.tiles_m : (live + kTile - 1) / kTile;
    const int32_t tn = q.tiles_n;
    const int64_t tiles = static_cast<int64_t>(tm) * tn * (MODE == kLinDh ? q.splits : 1);
    const int64_t pair0 = blockIdx.x >> 1, pairs_at_work = gridDim.x >> 1;
    const int32_t depth = MODE == kLinDw ? live : q.depth;
    const int32_t blocks_all = (depth + kDepth - 1) / kDepth;

    // depth blocks [first, last) of a tile
    const auto depth_first = [&](int32_t split) {
        return MODE == kLinDh ? static_cast<int32_t>(static_cast<int64_t>(blocks_all) * split / q.splits) : 0;
    };
    const auto depth_last = [&](int32_t split) {
        return MODE == kLinDh ? static_cast<int32_t>(static_cast<int64_t>(blocks_all) * (split + 1) / q.splits)
                              : blocks_all;
    };

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int64_t t = pair0; ok && t < tiles; t += pairs_at_work) {
                const TileId id = tile_of<MODE>(t, tm, tn);
                const int32_t k0 = depth_first(id.split), k1 = depth_last(id.split);
                const int32_t m0 = id.m * kTile + static_cast<int32_t>(rank) * 128;
                const int32_t n0 = id.n * kTile + static_cast<int32_t>(rank) * 128;
                for (int pr = 0; ok && pr < q.pairs; ++pr) {
                    const int za = plane_a(q.pairs, pr), zb = plane_b(q.pairs, pr);
                    for (int32_t kb = k0; kb < k1; ++kb) {
                        if (!wait_or_fail(&sh->empty[stage], phase ^ 1u, sh, q.dev_status)) {
                            ok = false;
                            break;
                        }
                        uint8_t *a = ring + stage * kStageBytes, *b = a + kHalfBytes;
                        if (rank == 0)
                            mbar_arrive_expect_tx(&sh->full[stage], 2 * kStageBytes);
                        const uint32_t bar = map_to_rank(smem_addr(&sh->full[stage]), 0);
                        const int32_t k = kb * kDepth;
                        if (MODE == kLinDw) {
                            tma_load_3d_pair(a, &map_a, m0, k, za, bar);
                            tma_load_3d_pair(a + kHalfBytes / 2, &map_a, m0 + 64, k, za, bar);
                        } else {
                            tma_load_3d_pair(a, &map_a, k, m0, za, bar);
                        }
                        if (MODE == kLinDw || MODE == kLinDh) {
                            const int32_t row = MODE == kLinDh ? q.b_row0 + k : k;
                            tma_load_3d_pair(b, &map_b, n0, row, zb, bar);
                            tma_load_3d_pair(b + kHalfBytes / 2, &map_b, n0 + 64, row, zb, bar);
                        } else {
                            tma_load_3d_pair(b, &map_b, k, q.b_row0 + n0, zb, bar);
                        }
                        if (++stage == kRing) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                }
            }
            // every stage used is free again: no copy is in flight and no
            // arrival is on its way to this CTA when it ends
            for (int i = 0; ok && i < kRing; ++i) {
                ok = wait_or_fail(&sh->empty[stage], phase ^ 1u, sh, q.dev_status);
                if (++stage == kRing) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            constexpr bool kAmn = MODE == kLinDw, kBmn = MODE == kLinDw || MODE == kLinDh;
            constexpr uint32_t idesc = mma_idesc(kTile, kTile, kAmn, kBmn);
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (int64_t t = pair0; ok && t < tiles; t += pairs_at_work) {
                const TileId id = tile_of<MODE>(t, tm, tn);
                const int32_t n_blocks = (depth_last(id.split) - depth_first(id.split)) * q.pairs;
                ok = wait_or_fail(&sh->acc_empty[acc], acc_phase ^ 1u, sh, q.dev_status);
                tc_fence_after();
                const uint32_t d = tmem + acc * kTile;
                for (int32_t kb = 0; ok && kb < n_blocks; ++kb) {
                    ok = wait_or_fail(&sh->full[stage], phase, sh, q.dev_status);
                    if (!ok)
                        break;
                    tc_fence_after();
                    const uint32_t a = smem_addr(ring + stage * kStageBytes), b = a + kHalfBytes;
#pragma unroll
                    for (int kk = 0; kk < kDepth / 16; ++kk) {
                        const uint64_t da = kAmn ? mma_desc(a + kk * 2048, kHalfBytes / 2, 1024)
                                                 : mma_desc(a + kk * 32, 16, 1024);
                        const uint64_t db = kBmn ? mma_desc(b + kk * 2048, kHalfBytes / 2, 1024)
                                                 : mma_desc(b + kk * 32, 16, 1024);
                        mma_bf16_pair(d, da, db, idesc, kb > 0 || kk > 0);
                    }
                    mma_commit_pair(&sh->empty[stage]);
                    if (++stage == kRing) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (ok)
                    mma_commit_pair(&sh->acc_full[acc]);
                acc ^= 1;
                acc_phase ^= acc == 0 ? 1u : 0u;
            }
        }
        __syncwarp();
    } else {
        const int quad = warp & 3;  // the TMEM lanes that this warp may read
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const int32_t tile_row = static_cast<int32_t>(rank) * 128 + quad * 32 + lane;
        const float alpha = MODE == kLinDw ? q.head->alpha : 1.0f;
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int64_t t = pair0; t < tiles; t += pairs_at_work) {
            const TileId id = tile_of<MODE>(t, tm, tn);
            const bool any = depth_last(id.split) > depth_first(id.split);
            const int32_t row = id.m * kTile + tile_row;
            const int64_t col0 = static_cast<int64_t>(id.n) * kTile;
            // stats, dz: this row's gathered columns, as bits of the tile
            uint32_t hit[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            bool any_hit = false;
            float2 g = make_float2(0.0f, 0.0f);
            if ((MODE == kLinStats || MODE == kLinDz) && row < live) {
                if (MODE == kLinDz)
                    g = q.grow[row];
                for (int k = 0; k < q.k; ++k) {
                    const int64_t j = q.tgt[static_cast<int64_t>(row) * q.k + k] - (q.v0 + col0);
                    if (j >= 0 && j < kTile) {
                        any_hit = true;
#pragma unroll
                        for (int w = 0; w < 8; ++w)
                            if (MODE == kLinStats && j >> 5 == w)
                                hit[w] |= 1u << (j & 31);
                    }
                }
            }
            if (!__all_sync(0xffffffffu, wait_or_fail(&sh->acc_full[acc], acc_phase, sh, q.dev_status)))
                break;
            tc_fence_after();
            const uint32_t src = tmem + lanes + acc * kTile;
            RowStats st;
#pragma unroll 1
            for (int ch = 0; ch < kTile / 32; ++ch) {
                float v[32];
                tmem_load32(src + ch * 32, v);
                if (ch == kTile / 32 - 1) {  // the sums are read: the tile after next may start
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive_remote(map_to_rank(smem_addr(&sh->acc_empty[acc]), 0));
                }
                const int64_t c0 = col0 + ch * 32;
                if (MODE == kLinStats) {
                    const int64_t end = q.vocab - (q.v0 + c0);  // columns of this chunk that exist
                    if (end < 32) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            v[j] = j < end ? v[j] : kNegInf;
                    }
                    uint32_t mine = 0;
#pragma unroll
                    for (int w = 0; w < 8; ++w)
                        mine = ch == w ? hit[w] : mine;
                    if (mine != 0) {
                        for (int k = 0; k < q.k; ++k) {
                            const int64_t at = static_cast<int64_t>(row) * q.k + k;
                            const int64_t j = q.tgt[at] - (q.v0 + c0);
                            if (j >= 0 && j < 32) {
                                float x = v[0];
#pragma unroll
                                for (int i = 1; i < 32; ++i)
                                    x = j == i ? v[i] : x;
                                q.xt[at] = x;
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            v[j] = mine >> j & 1u ? kNegInf : v[j];
                    }
                    st.add(v, q.c);
                }
                if (MODE == kLinDz) {
                    const int64_t end = q.vocab - (q.v0 + c0);
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[j] = row < live && j < end ? g.y * ex2((v[j] - g.x) * q.c) : 0.0f;
                    __nv_bfloat16 *out = q.dz + static_cast<int64_t>(row) * q.piece + c0;
                    for (int z = 0; z < q.planes; ++z, out += q.dz_plane) {
#pragma unroll
                        for (int j = 0; j < 32; j += 8) {
                            uint4 w;
                            w.x = pack_bf16(v[j], v[j + 1]);
                            w.y = pack_bf16(v[j + 2], v[j + 3]);
                            w.z = pack_bf16(v[j + 4], v[j + 5]);
                            w.w = pack_bf16(v[j + 6], v[j + 7]);
                            *reinterpret_cast<uint4 *>(out + j) = w;
                            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 f = bf16x2_to_float2(ws[i]);
                                v[j + 2 * i] -= f.x;
                                v[j + 2 * i + 1] -= f.y;
                            }
                        }
                    }
                }
                if (MODE == kLinDh && row < live) {
                    float *out = q.dh + static_cast<int64_t>(id.split) * q.dh_split +
                                 static_cast<int64_t>(row) * q.dh_pitch + c0;
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        if (c0 + j < q.dim) {
                            float4 x = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                            if (!any)
                                x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            if (!q.first) {
                                const float4 old = *reinterpret_cast<const float4 *>(out + j);
                                x = make_float4(old.x + x.x, old.y + x.y, old.z + x.z, old.w + x.w);
                            }
                            *reinterpret_cast<float4 *>(out + j) = x;
                        }
                }
                if (MODE == kLinDw && q.v0 + row < q.vocab) {
                    const int64_t at = (q.v0 + row) * q.dweight_stride + c0;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[j] = any ? alpha * v[j] : 0.0f;
                    const bool whole = q.vec != 0 && c0 + 32 <= q.dim;
                    if (q.bf16) {
                        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(q.dweight) + at;
                        if (whole) {
#pragma unroll
                            for (int j = 0; j < 32; j += 8) {
                                uint4 *o = reinterpret_cast<uint4 *>(out + j);
                                if (q.accumulate) {
                                    const uint4 old = *o;
                                    const uint32_t ow[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        const float2 f = bf16x2_to_float2(ow[i]);
                                        v[j + 2 * i] += f.x;
                                        v[j + 2 * i + 1] += f.y;
                                    }
                                }
                                *o = make_uint4(pack_bf16(v[j], v[j + 1]), pack_bf16(v[j + 2], v[j + 3]),
                                                pack_bf16(v[j + 4], v[j + 5]), pack_bf16(v[j + 6], v[j + 7]));
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (c0 + j < q.dim)
                                    out[j] = __float2bfloat16_rn(
                                        q.accumulate ? __bfloat162float(out[j]) + v[j] : v[j]);
                        }
                    } else {
                        float *out = static_cast<float *>(q.dweight) + at;
                        if (whole) {
#pragma unroll
                            for (int j = 0; j < 32; j += 4) {
                                float4 *o = reinterpret_cast<float4 *>(out + j);
                                float4 x = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                                if (q.accumulate) {
                                    const float4 old = *o;
                                    x = make_float4(old.x + x.x, old.y + x.y, old.z + x.z, old.w + x.w);
                                }
                                *o = x;
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (c0 + j < q.dim)
                                    out[j] = q.accumulate ? out[j] + v[j] : v[j];
                        }
                    }
                }
            }
            if (MODE == kLinStats && row < live)
                q.partials[static_cast<int64_t>(row) * q.partial_tiles + q.v0 / kTile + id.n] =
                    make_float2(st.s == st.s ? st.m : (st.m == kNegInf ? 0.0f : st.m), st.s);
            if (MODE == kLinDz && any_hit) {
                // the gathered columns, over what this thread wrote above
                for (int k = 0; k < q.k; ++k) {
                    const int64_t at = static_cast<int64_t>(row) * q.k + k;
                    const int64_t j = q.tgt[at] - (q.v0 + col0);
                    if (j >= 0 && j < kTile) {
                        float x = q.dzt[at];
                        __nv_bfloat16 *out = q.dz + static_cast<int64_t>(row) * q.piece + col0 + j;
                        for (int z = 0; z < q.planes; ++z, out += q.dz_plane) {
                            const __nv_bfloat16 w = __float2bfloat16_rn(x);
                            *out = w;
                            x -= __bfloat162float(w);
                        }
                    }
                }
            }
            acc ^= 1;
            acc_phase ^= acc == 0 ? 1u : 0u;
        }
        __syncwarp();
    }

    // Past a wait that gave up, copies and products may be in flight: they
    // get a millisecond before their memory goes.
    __syncthreads();
    if (*reinterpret_cast<volatile int32_t *>(&sh->failed) != 0)
        for (int i = 0; i < 1000; ++i)
            __nanosleep(1000);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_free_pair(tmem, kTmemCols);
    }
    __syncthreads();
    cluster_sync();
}

// ----------------------------------------------------------------- launches

namespace {

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                              const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                              const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once per process.
EncodeFn encoder()
{
    static EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// bf16 planes of [rows, inner], rows `stride` and planes `plane` elements
// apart, read in boxes of 64 x box_rows with the 128-byte swizzle; what lies
// outside reads as zeros.
cudaError_t make_map(CUtensorMap *map, const void *base, int64_t inner, int64_t rows, int64_t stride,
                     int64_t planes, int64_t plane, uint32_t box_rows)
{
    const EncodeFn fn = encoder();
    if (fn == nullptr)
        return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(planes)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(stride) * 2,
                                   static_cast<cuuint64_t>(plane) * 2};
    const cuuint32_t box[3] = {64, box_rows, 1}, step[3] = {1, 1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims,
                          strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int MODE>
cudaError_t launch_mma(const CUtensorMap &a, const CUtensorMap &b, const MmaArgs &q, int64_t max_tiles,
                       cudaStream_t s)
{
    const int sms = device_sm_count();
    if (sms < 2)
        return cudaErrorInvalidDevice;
    cudaError_t e = cudaFuncSetAttribute(lin_mma_kernel<MODE>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess)
        return e;
    const int64_t pairs = max_tiles < sms / 2 ? max_tiles : sms / 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
    cfg.blockDim = dim3(kMmaThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, lin_mma_kernel<MODE>, a, b, q);
    note_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// What the logits' operands look like to the kernels for one piece.
struct Weight {
    const void *base;
    int64_t rows, stride, plane;  // of the map
    int64_t row0;                 // the piece's first row in it
};

// `packed`: an earlier launch of the call has been here.
cudaError_t piece_weight(const LinParams &p, int64_t v0, int64_t v1, bool packed, Weight &w,
                         cudaStream_t s)
{
    if (p.weight_direct) {
        w = {p.weight, p.vocab, p.weight_stride, p.weight_stride, v0};  // one plane
        return cudaSuccess;
    }
    const bool whole = p.wpack_rows >= p.vocab;  // packed once for every use
    w = {p.wpack, whole ? p.vocab : v1 - v0, p.pitch, p.wpack_rows * p.pitch, whole ? v0 : 0};
    if (whole && packed)
        return cudaSuccess;
    return whole ? lin_pack_weight(p, 0, p.vocab, s) : lin_pack_weight(p, v0, v1, s);
}

MmaArgs base_args(const LinParams &p, int64_t v0)
{
    MmaArgs q{};
    q.head = p.head;
    q.dev_status = p.dev_status;
    q.planes = p.planes;
    q.pairs = p.planes == 1 ? 1 : 6;
    q.splits = 1;
    q.v0 = v0;
    q.vocab = p.vocab;
    q.c = p.c;
    q.k = static_cast<int32_t>(p.k);
    q.tgt = p.tgt;
    q.dim = p.dim;
    return q;
}

int64_t tiles_of(int64_t n) { return (n + kTile - 1) / kTile; }

}  // namespace

cudaError_t lin_stats(const LinParams &p, cudaStream_t s)
{
    const int64_t step = p.weight_direct ? p.vocab : p.wpack_rows;
    for (int64_t v0 = 0; v0 < p.vocab; v0 += step) {
        const int64_t v1 = v0 + step < p.vocab ? v0 + step : p.vocab;
        Weight w;
        cudaError_t e = piece_weight(p, v0, v1, v0 > 0, w, s);
        CUtensorMap a, b;
        if (e == cudaSuccess)
            e = make_map(&a, p.hpack, p.dim, p.rows, p.pitch, p.planes, p.hpack_plane, 128);
        if (e == cudaSuccess)
            e = make_map(&b, w.base, p.dim, w.rows, w.stride, p.planes, w.plane, 128);
        if (e != cudaSuccess)
            return e;
        MmaArgs q = base_args(p, v0);
        q.depth = static_cast<int32_t>(p.dim);
        q.tiles_n = static_cast<int32_t>(tiles_of(v1 - v0));
        q.b_row0 = static_cast<int32_t>(w.row0);
        q.xt = p.xt;
        q.partials = p.partials;
        q.partial_tiles = p.tiles;
        e = launch_mma<kLinStats>(a, b, q, tiles_of(p.rows) * q.tiles_n, s);
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

cudaError_t lin_grads(const LinParams &p, cudaStream_t s)
{
    for (int64_t v0 = 0; v0 < p.vocab; v0 += p.piece) {
        const int64_t v1 = v0 + p.piece < p.vocab ? v0 + p.piece : p.vocab;
        Weight w;
        cudaError_t e = piece_weight(p, v0, v1, v0 > 0 || p.fused, w, s);
        CUtensorMap h_k, w_k, dz_k, w_mn, dz_mn, h_mn;
        const auto map = [&e](CUtensorMap *m, const void *base, int64_t inner, int64_t rows,
                              int64_t stride, int64_t planes, int64_t plane, uint32_t box) {
            if (e == cudaSuccess)
                e = make_map(m, base, inner, rows, stride, planes, plane, box);
        };
        map(&h_k, p.hpack, p.dim, p.rows, p.pitch, p.planes, p.hpack_plane, 128);
        map(&h_mn, p.hpack, p.dim, p.rows_pad, p.pitch, p.planes, p.hpack_plane, 64);
        map(&w_k, w.base, p.dim, w.rows, w.stride, p.planes, w.plane, 128);
        map(&w_mn, w.base, p.dim, w.rows, w.stride, p.planes, w.plane, 64);
        map(&dz_k, p.dz, p.piece, p.rows_pad, p.piece, p.planes, p.dz_plane, 128);
        map(&dz_mn, p.dz, p.piece, p.rows_pad, p.piece, p.planes, p.dz_plane, 64);
        if (e != cudaSuccess)
            return e;
        const int64_t tv = tiles_of(v1 - v0), td = tiles_of(p.dim), tr = tiles_of(p.rows);
        MmaArgs q = base_args(p, v0);
        q.b_row0 = static_cast<int32_t>(w.row0);
        q.grow = p.grow;
        q.dzt = p.dzt;
        q.dz = static_cast<__nv_bfloat16 *>(p.dz);
        q.piece = p.piece;
        q.dz_plane = p.dz_plane;
        q.depth = static_cast<int32_t>(p.dim);
        q.tiles_n = static_cast<int32_t>(tv);
        e = launch_mma<kLinDz>(h_k, w_k, q, tr * tv, s);
        q.tiles_n = static_cast<int32_t>(td);
        if (e == cudaSuccess && p.dhidden != nullptr) {
            q.depth = static_cast<int32_t>(v1 - v0);
            q.splits = p.dh_splits;
            q.first = v0 == 0;
            q.dh = p.dh;
            q.dh_pitch = p.dh_pitch;
            q.dh_split = p.rows_pad * p.dh_pitch;
            e = launch_mma<kLinDh>(dz_k, w_mn, q, tr * td * p.dh_splits, s);
        }
        if (e == cudaSuccess && p.dweight != nullptr) {
            const size_t es = p.bf16 ? 2 : 4;
            q.tiles_m = static_cast<int32_t>(tv);
            q.dweight = p.dweight;
            q.dweight_stride = p.dweight_stride;
            q.accumulate = p.accumulate;
            q.bf16 = p.bf16;
            q.vec = reinterpret_cast<uintptr_t>(p.dweight) % 16 == 0 &&
                    static_cast<size_t>(p.dweight_stride) * es % 16 == 0;
            e = launch_mma<kLinDw>(dz_mn, h_mn, q, tv * td, s);
        }
        if (e != cudaSuccess)
            return e;
    }
    return p.dhidden == nullptr ? cudaSuccess : lin_finish(p, s);
}

}  // namespace gbce
