// The matrix products of the calls that start from hidden states, on the
// tensor cores: one kernel, three uses.
//
//   stats  logits = hidden . weight^T    -> (max, sum) per row and tile
//   dz     the same logits again         -> dz, in memory for one piece
//   grads  dz . weight                   -> dhidden sums (fp32), and in the
//          dz^T . hidden                 -> same launch dweight rows of the piece
//
// TMA brings 64-deep slices of both operands of a tile into a ring, one thread
// issues the MMAs, and the sums lie in TMEM, two tiles' worth, so that eight
// warps turn one tile into outputs while the next is multiplied.  Persistent:
// every CTA (or pair of CTAs) takes tiles until there are no more.
//
// Tiles.  256 x 256 by a pair of CTAs (M = 256 across the pair, each loads
// half of both operands) moves the fewest bytes per product and is what large
// calls run.  128 x {256, 128, 64} by single CTAs is for calls whose 256 x 256
// tiles would leave SMs idle, and, 256 wide, for up to 128 rows, where the
// weight's bytes are the work and half of a pair's rows would be empty.
// choose_tile() takes the shape with the least estimated time.
//
// Operands are read in the layout they have: hidden, weight and dz lie with
// the product's depth innermost for the logits (and dz for dhidden), and with
// it outermost for dhidden's weight and both operands of dweight; the matrix
// descriptors take either, so that nothing is ever transposed in memory.
//
// fp32 inputs come as three bf16 planes, x = hi + mid + lo with 8 more bits
// in each; six of the nine products (all above 2^-24 of x y) are summed,
// smallest first, so that the large ones meet a sum that is still small.
//
// dz of bf16 inputs is one bf16 plane, rounded once, as dlogits of bf16 logits
// are.  In two planes (16 bits) the gradients' error against 64 bits is that of
// their own rounding, 1.66e-3 in norm; in one it is 1.68e-3 to 1.71e-3 where
// many rows' dz meet (losses of 256 to 613 rows) and 2.4e-3 where one gathered
// column leads each row's (log-probs of 2048 x 151936).  The second plane
// doubles both gradients' products: 8192 x 152064 x 4096 23.4 -> 35.6 ms, 2048
// x 151936 x 2560 with its forward 3.5 -> 5.4, 613 x 40001 x 1001 256 -> 326 us.
#include <atomic>

#include <cuda.h>

#include "gbce_kernels.cuh"
#include "gbce_linear.h"
#include "gbce_linear_rows.cuh"
#include "gbce_umma.cuh"

namespace gbce {

namespace {

constexpr int kDepth = 64;           // depth of a stage: 128 bytes of bf16
constexpr uint32_t kRowBytes = kDepth * 2;
constexpr uint32_t kBytesA = 128 * kRowBytes;  // a CTA's rows of A in a stage
constexpr int kMmaThreads = 320;     // TMA warp, MMA warp, eight epilogue warps

// kLinGradsSplit: grads of operands in planes (fp32), summed in segments.
enum LinMode : int { kLinStats, kLinDz, kLinGrads, kLinGradsSplit };

__host__ __device__ constexpr bool is_grads(int mode) { return mode >= kLinGrads; }

// Blocks of depth in one sum of the tensor cores.  They cut each partial sum's
// last bits rather than round them, so a sum of many steps comes out small by
// a part that grows with their number.  Logits are therefore summed 1024 deep
// at a time (256 for up to 128 rows, where the table's bytes leave the time),
// the gradients of fp32 inputs 512 deep, and these sums added in fp32
// registers, rounded to nearest; those of bf16 gradients, which end in 8 bits,
// are one sum.  Log-probs of 7000 x 76032 x 2560, relative error: 1.2e-6 in
// one sum, 3.9e-7 1024 deep, 2.1e-7 512 deep (in fp32 products 2e-7 to 4e-7);
// loss and gradients 5.87 ms 1024 deep, 6.22 512 deep.  dhidden of 2000 x 60000
// x 512 fp32: 1.1e-6 1024 deep, 6.4e-7 512 deep (fp32 products 5.1e-6); 5% of
// the time.
//
// The gathered columns' own logits are not taken from these sums: a row whose
// target leads by 45 has a log p of e^-45 whose relative error is the absolute
// error of that logit, and a logit of 50 summed 1024 deep came out 4e-5 too
// small.  They are fp32 products of their two rows (row_dot), made apart: such
// rows' log p is then within 2e-7 (1 x 152064 x 4096).  What that costs: 2048
// x 32768 x 1024 92 -> 98 us, 7000 x 76032 x 2560 nothing.
constexpr int kSegLogits = 16, kSegShort = 4, kSegGrads = 8;

template <int CTAS, int NT> struct Tile {
    static constexpr int kM = 128 * CTAS;
    static constexpr int kRowsB = NT / CTAS;  // rows of B that a CTA loads
    static constexpr uint32_t kBytesB = kRowsB * kRowBytes;
    static constexpr uint32_t kStage = kBytesA + kBytesB;
    static constexpr int kRing = 196608 / kStage;  // 6, 4, 6 or 8 stages
    static constexpr uint32_t kTmemCols = 2 * NT;
};

struct MmaArgs {
    LinHeader *head;
    int32_t *dev_status;
    int32_t pairs;         // plane products: 1, or 6 for fp32 inputs
    int32_t blocks;        // stats, dz, dhidden: the depth in blocks of kDepth
    int32_t tiles_n;       // stats, dz: of the piece; grads: of dim
    int32_t tiles_v;       // grads: tiles of the piece's rows (0: no dweight)
    int32_t want_dh;
    int32_t piece_blocks;  // grads: blocks of a whole piece
    int32_t units;         // grads: CTAs or pairs that the GPU holds
    int32_t a_rows;        // stats, dz: rows of A's box
    int32_t b_row0;        // the piece's first row in the weight's map
    int64_t v0, vocab;     // first column of the piece; end of the vocabulary
    float c;
    int32_t k;
    const int32_t *tgt;
    const int64_t *targets;  // stats of a direct call: [direct_rows, k]
    int32_t direct_rows;     // else 0
    int32_t seg;                  // stats, dz: blocks of a segment
    const void *hidden, *weight;  // stats: for the gathered columns' logits
    int64_t hidden_stride, weight_stride;
    const int32_t *row_list;
    float *xt;
    float2 *partials;
    int64_t partial_tiles;
    float *z;              // stats: keep the logits here, rows z_pitch apart
    int64_t z_pitch;
    const float2 *grow;
    const float *dzt;
    __nv_bfloat16 *dz;
    int64_t piece, dz_plane;
    int32_t planes;
    float *dh;
    int64_t dim, dh_pitch, dh_room;
    void *dweight;
    int64_t dweight_stride;
    int32_t first, accumulate, bf16;
    int32_t vec;           // dweight's rows start on so many bytes: 32, 16 or 0 (fewer)
};

template <int RING> struct MmaShared {
    uint64_t full[RING], empty[RING], acc_full[2], acc_empty[2];
    uint32_t tmem;
    int32_t failed;
    float turn[8][32][33];  // a warp's 32 x 32 values, to be stored by rows
};

template <int CTAS, int NT>
constexpr uint32_t smem_bytes()
{
    using S = Tile<CTAS, NT>;
    return S::kRing * S::kStage + sizeof(MmaShared<S::kRing>) + 1024;
}

// One tile's work: which operands, where, and how deep.
struct Job {
    int32_t m, n, split;
    int32_t k0, k1;  // depth blocks
    bool dw;         // grads: a dweight tile, else a dhidden tile
};

// The tiles of a launch, the same for every role.
template <int MODE> struct Jobs {
    int32_t tm, tn, tv, splits, blocks, live_blocks;
    int64_t dh_tiles, total;

    __device__ Jobs(const MmaArgs &q, int32_t live, int tile_m)
    {
        tm = (live + tile_m - 1) / tile_m;
        tn = q.tiles_n;
        blocks = q.blocks;
        splits = 1;
        tv = 0;
        live_blocks = (live + kDepth - 1) / kDepth;
        if (!is_grads(MODE)) {
            dh_tiles = total = static_cast<int64_t>(tm) * tn;
            return;
        }
        tv = q.tiles_v;
        dh_tiles = q.want_dh ? static_cast<int64_t>(tm) * tn : 0;
        // dhidden's depth, the vocabulary, is split into parts of equal depth
        // where its tiles would not come out even over the CTAs (80 tiles for
        // 76 pairs are two turns, in eight parts 8.4 of 9).  A part costs about
        // 24 products of 64 deep: its sums go to memory.  2048 x 77824 x 2560:
        // 1055 TFLOP/s whole, 1587 split.  The same for every piece of a call,
        // whose sums are added, and whether or not dweight is wanted.
        // Each lane looks at two numbers of parts.
        if (dh_tiles > 0) {
            const float room = static_cast<float>(q.dh_room / (static_cast<int64_t>(tm) * tile_m * q.dh_pitch));
            const float n = static_cast<float>(dh_tiles), u = static_cast<float>(q.units);
            const float depth = static_cast<float>(q.piece_blocks);
            const float extra = 24.0f / static_cast<float>(q.pairs);
            uint32_t least = 0xffffffffu, mine = 1;  // costs are positive: their bits compare alike
#pragma unroll
            for (uint32_t k = (threadIdx.x & 31) + 1; k <= kMaxSplits; k += 32) {
                const float parts = static_cast<float>(k), part = depth / parts + extra;
                const uint32_t cost = __float_as_uint(ceilf(n * parts / u) * part + parts / static_cast<float>(q.pairs));
                if (cost < least && (k == 1 || parts <= room)) {
                    least = cost;
                    mine = k;
                }
            }
            const uint32_t best = __reduce_min_sync(0xffffffffu, least);
            splits = static_cast<int32_t>(__reduce_min_sync(0xffffffffu, least == best ? mine : kMaxSplits));
        }
        dh_tiles *= splits;
        total = dh_tiles + static_cast<int64_t>(tv) * tn;
    }

    // Tiles in an order that keeps both operands in L2 while they are needed.
    // Logits: all row tiles (hidden stays in L2) before the next columns, so
    // that the table is read once.  Gradients: bands of 8 tiles high, so that
    // the CTAs at work cover a block that is about square; dhidden's first,
    // being the deeper ones.
    __device__ __forceinline__ Job at(int64_t t) const
    {
        Job j;
        j.split = 0;
        j.dw = false;
        j.k0 = 0;
        j.k1 = blocks;
        if (!is_grads(MODE)) {
            j.m = static_cast<int32_t>(t % tm);
            j.n = static_cast<int32_t>(t / tm);
            return j;
        }
        int32_t high_all = tm;
        if (t >= dh_tiles) {
            t -= dh_tiles;
            j.dw = true;
            j.k1 = live_blocks;
            high_all = tv;
        } else {
            const int64_t per = static_cast<int64_t>(tm) * tn;
            j.split = static_cast<int32_t>(t / per);
            t %= per;
            j.k0 = static_cast<int32_t>(static_cast<int64_t>(blocks) * j.split / splits);
            j.k1 = static_cast<int32_t>(static_cast<int64_t>(blocks) * (j.split + 1) / splits);
        }
        const int32_t u = static_cast<int32_t>(t);
        const int32_t band = u / (8 * tn), in = u % (8 * tn);
        const int32_t high = min(8, high_all - band * 8);
        j.m = band * 8 + in % high;
        j.n = in / high;
        return j;
    }
};

// Column of a row's k-th target, from column 0 of the tile; out of the tile's
// range for a target out of the vocabulary's.
__device__ __forceinline__ int64_t target_column(const MmaArgs &q, int64_t at, int64_t first)
{
    if (q.direct_rows == 0)
        return q.tgt[at] - first;
    const int64_t t = q.targets[at];
    return t < 0 || t >= q.vocab ? -1 : t - first;
}

// Logit of gathered column `at` (row x k + target), by a warp.
__device__ __forceinline__ void target_logit(const MmaArgs &q, int64_t at)
{
    const int64_t t = target_column(q, at, 0), i = at / q.k;
    if (t < 0)
        return;
    const int64_t r = q.direct_rows == 0 ? q.row_list[i] : i;
    float x;
    if (q.planes == 1)
        x = row_dot(static_cast<const __nv_bfloat16 *>(q.hidden) + r * q.hidden_stride,
                    static_cast<const __nv_bfloat16 *>(q.weight) + t * q.weight_stride, q.dim);
    else
        x = row_dot(static_cast<const float *>(q.hidden) + r * q.hidden_stride,
                    static_cast<const float *>(q.weight) + t * q.weight_stride, q.dim);
    if ((threadIdx.x & 31) == 0)
        q.xt[at] = x;
}

// Plane indices of product q of six, smallest first.
__device__ __forceinline__ int plane_a(int pairs, int q) { return pairs == 1 ? 0 : (0x201100 >> (4 * (5 - q))) & 15; }
__device__ __forceinline__ int plane_b(int pairs, int q) { return pairs == 1 ? 0 : (0x021010 >> (4 * (5 - q))) & 15; }

__device__ __forceinline__ bool wait_or_fail(uint64_t *bar, uint32_t parity, int32_t *failed,
                                             int32_t *dev_status)
{
    if (mbar_wait(bar, parity))
        return true;
    *reinterpret_cast<volatile int32_t *>(failed) = 1;
    report(dev_status, GBCE_DEV_TIMEOUT);
    return false;
}

// The same for a whole warp, which goes on or gives up together.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, int32_t *failed,
                                          int32_t *dev_status)
{
    return __all_sync(0xffffffffu, wait_or_fail(bar, parity, failed, dev_status));
}

// ------------------------------------------------------------- epilogues

// Running (max, sum) over the columns that one thread has of its row.
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

// One thread's 32 columns of a row, which starts on 16 bytes (`wide`: on 32).
__device__ __forceinline__ void store_row(__nv_bfloat16 *out, float (&v)[32], bool accumulate, bool wide)
{
#pragma unroll
    for (int j = 0; j < 32; j += 16) {
        uint4 *o = reinterpret_cast<uint4 *>(out + j);
        if (accumulate) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 old = o[h];
                const uint32_t ow[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = bf16x2_to_float2(ow[i]);
                    v[j + 8 * h + 2 * i] += f.x;
                    v[j + 8 * h + 2 * i + 1] += f.y;
                }
            }
        }
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = pack_bf16(v[j + 2 * i], v[j + 2 * i + 1]);
        if (wide) {
            st_v8(static_cast<void *>(o), w);
        } else {
            o[0] = make_uint4(w[0], w[1], w[2], w[3]);
            o[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
}

__device__ __forceinline__ void store_row(float *out, float (&v)[32], bool accumulate, bool wide)
{
#pragma unroll
    for (int j = 0; j < 32; j += 8) {
        float4 *o = reinterpret_cast<float4 *>(out + j);
        if (accumulate) {
            const float4 a = o[0], b = o[1];
            v[j] += a.x, v[j + 1] += a.y, v[j + 2] += a.z, v[j + 3] += a.w;
            v[j + 4] += b.x, v[j + 5] += b.y, v[j + 6] += b.z, v[j + 7] += b.w;
        }
        if (wide) {
            st_v8(out + j, v + j);
        } else {
            o[0] = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
            o[1] = make_float4(v[j + 4], v[j + 5], v[j + 6], v[j + 7]);
        }
    }
}

// Stores of one 32 x 32 block whose rows do not start on 16 bytes: through
// shared memory, so that a warp writes one row's 32 columns at a time.
template <typename T>
__device__ __forceinline__ void store_rows_turned(float (&buf)[32][33], const float (&v)[32], T *out,
                                                  int64_t stride, int32_t rows, int32_t cols,
                                                  bool accumulate)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 32; ++j)
        buf[lane][j] = v[j];
    __syncwarp();
    if (lane < cols) {
#pragma unroll 8
        for (int r = 0; r < rows; ++r) {
            T *o = out + r * stride + lane;
            const float x = buf[r][lane];
            *o = T(accumulate ? static_cast<float>(*o) + x : x);
        }
    }
    __syncwarp();
}

template <int MODE, int CTAS, int NT>
__global__ void __launch_bounds__(kMmaThreads, 1)
    lin_mma_kernel(const __grid_constant__ CUtensorMap map_a,
                   const __grid_constant__ CUtensorMap map_b,
                   const __grid_constant__ CUtensorMap map_a2,
                   const __grid_constant__ CUtensorMap map_b2, const __grid_constant__ MmaArgs q)
{
    using S = Tile<CTAS, NT>;
    constexpr int kRing = S::kRing;
    extern __shared__ uint8_t raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t{1023});
    MmaShared<kRing> *sh = reinterpret_cast<MmaShared<kRing> *>(ring + kRing * S::kStage);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CTAS == 2 ? cluster_rank() : 0;
    if (threadIdx.x == 0) {
        tma_prefetch_map(&map_a);
        tma_prefetch_map(&map_b);
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&sh->full[i], 1);
            mbar_init(&sh->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->acc_full[i], 1);
            mbar_init(&sh->acc_empty[i], 8 * CTAS);  // eight warps of each CTA
        }
        sh->failed = 0;
        fence_barrier_init();
    }
    if (warp == 1)
        tmem_alloc<CTAS>(&sh->tmem, S::kTmemCols);
    tc_fence_before();
    __syncthreads();
    if (CTAS == 2)
        cluster_sync();  // both CTAs' barriers exist before either signals them
    tc_fence_after();
    const uint32_t tmem = sh->tmem;

    grid_dependency_wait();
    launch_dependents();
    const int32_t live = q.direct_rows > 0 ? q.direct_rows : q.head->n_live;
    if (MODE == kLinStats && q.direct_rows > 0 && blockIdx.x == 0 && threadIdx.x == 0) {
        q.head->n_live = live;
        q.head->n_items = 0;  // the combine counts
        q.head->done = 0;
    }
    const int64_t units = gridDim.x / CTAS, unit = blockIdx.x / CTAS;
    const Jobs<MODE> jobs(q, live, S::kM);
    if (is_grads(MODE) && blockIdx.x == 0 && threadIdx.x == 0)
        q.head->dh_splits = jobs.splits;

    // The first two warps run whole, so that addresses and descriptors stay in
    // uniform registers, and elect the lane that issues: with one lane in the
    // loop a stage took some 540 cycles to issue, more than a 128-wide tile's
    // products take.
    if (warp == 0) {
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int64_t t = unit; ok && t < jobs.total; t += units) {
            const Job job = jobs.at(t);
            const int32_t m0 = job.m * S::kM + static_cast<int32_t>(rank) * 128;
            const int32_t n0 = job.n * NT + static_cast<int32_t>(rank) * S::kRowsB;
            // bytes of a stage: A's box may be lower than the tile
            const uint32_t bytes = is_grads(MODE)
                                       ? S::kStage
                                       : static_cast<uint32_t>(q.a_rows) * kRowBytes + S::kBytesB;
            for (int pr = 0; ok && pr < q.pairs; ++pr) {
                const int za = plane_a(q.pairs, pr), zb = plane_b(q.pairs, pr);
                for (int32_t kb = job.k0; kb < job.k1; ++kb) {
                    ok = warp_wait(&sh->empty[stage], phase ^ 1u, &sh->failed, q.dev_status);
                    if (!ok)
                        break;
                    if (elect_one()) {
                        uint8_t *a = ring + stage * S::kStage, *b = a + kBytesA;
                        if (rank == 0)
                            mbar_arrive_expect_tx(&sh->full[stage], CTAS * bytes);
                        const uint32_t own = smem_addr(&sh->full[stage]);
                        const uint32_t bar = CTAS == 2 ? map_to_rank(own, 0) : own;
                        const int32_t k = kb * kDepth;
                        if (is_grads(MODE)) {
                            if (job.dw) {
                                tma_load_3d<CTAS>(a, &map_a2, m0, k, za, bar);
                                tma_load_3d<CTAS>(a + kBytesA / 2, &map_a2, m0 + 64, k, za, bar);
                            } else {
                                tma_load_3d<CTAS>(a, &map_a, k, m0, za, bar);
                            }
                            const CUtensorMap *mb = job.dw ? &map_b2 : &map_b;
                            const int32_t row = job.dw ? k : q.b_row0 + k;
#pragma unroll
                            for (int i = 0; i < S::kRowsB / 64; ++i)
                                tma_load_3d<CTAS>(b + i * 64 * kRowBytes, mb, n0 + 64 * i, row, zb, bar);
                        } else {
                            tma_load_3d<CTAS>(a, &map_a, k, m0, za, bar);
                            tma_load_3d<CTAS>(b, &map_b, k, q.b_row0 + n0, zb, bar);
                        }
                    }
                    __syncwarp();
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
            ok = warp_wait(&sh->empty[stage], phase ^ 1u, &sh->failed, q.dev_status);
            if (++stage == kRing) {
                stage = 0;
                phase ^= 1u;
            }
        }
    } else if (warp == 1) {
        if (rank == 0) {
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (int64_t t = unit; ok && t < jobs.total; t += units) {
                const Job job = jobs.at(t);
                const bool a_mn = is_grads(MODE) && job.dw, b_mn = is_grads(MODE);
                const uint32_t idesc = mma_idesc(S::kM, NT, a_mn, b_mn);
                // 16 deep: 32 bytes along a row, or two groups of 8 k-rows
                const uint32_t step_a = a_mn ? 2048 : 32, step_b = b_mn ? 2048 : 32;
                const int32_t n_blocks = (job.k1 - job.k0) * q.pairs;
                const int32_t seg = MODE == kLinGrads ? max(n_blocks, 1) : (is_grads(MODE) ? kSegGrads : q.seg);
                int32_t kb = 0;
                do {  // one sum in TMEM for each segment
                    ok = warp_wait(&sh->acc_empty[acc], acc_phase ^ 1u, &sh->failed, q.dev_status);
                    tc_fence_after();
                    const uint32_t d = tmem + acc * NT;
                    const int32_t k_end = min(n_blocks, kb + seg);
                    for (bool begun = false; ok && kb < k_end; ++kb, begun = true) {
                        ok = warp_wait(&sh->full[stage], phase, &sh->failed, q.dev_status);
                        if (!ok)
                            break;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint32_t a = smem_addr(ring + stage * S::kStage), b = a + kBytesA;
                            uint64_t da = mma_desc(a, 64 * kRowBytes, 8 * kRowBytes);
                            uint64_t db = mma_desc(b, 64 * kRowBytes, 8 * kRowBytes);
#pragma unroll
                            for (int kk = 0; kk < kDepth / 16; ++kk) {
                                mma_bf16<CTAS>(d, da, db, idesc, begun || kk > 0);
                                da += step_a >> 4;
                                db += step_b >> 4;
                            }
                            mma_commit<CTAS>(&sh->empty[stage]);
                        }
                        __syncwarp();
                        if (++stage == kRing) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    if (ok && elect_one())
                        mma_commit<CTAS>(&sh->acc_full[acc]);
                    __syncwarp();
                    acc ^= 1;
                    acc_phase ^= acc == 0 ? 1u : 0u;
                } while (ok && kb < n_blocks);
            }
        }
    } else {
        // A warp may read the 32 TMEM lanes that its number says; two share
        // them, each with half of the tile's columns.
        constexpr int kHalf = NT / 2, kChunks = kHalf / 32;
        const int quad = warp & 3, half = (warp - 2) >> 2;
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const int32_t warp_row = static_cast<int32_t>(rank) * 128 + quad * 32;
        const float alpha = is_grads(MODE) ? q.head->alpha : 1.0f;
        int acc = 0;
        uint32_t acc_phase = 0;
        // stats: this warp's share of the gathered columns' logits, the first
        // ones by different CTAs, before its tiles (more than one a warp, which
        // calls in place have where tiles are few: after them)
        const int64_t all_dots = MODE == kLinStats && q.xt != nullptr ? static_cast<int64_t>(live) * q.k : 0;
        const int64_t dot_step = static_cast<int64_t>(gridDim.x) * 8;
        int64_t dot = static_cast<int64_t>(warp - 2) * gridDim.x + blockIdx.x;
        const auto make_dots = [&] {
            for (; dot < all_dots; dot += dot_step)
                target_logit(q, dot);
        };
        if (MODE == kLinStats && all_dots <= dot_step)
            make_dots();
        for (int64_t t = unit; t < jobs.total; t += units) {
            const Job job = jobs.at(t);
            const bool any = job.k1 > job.k0;
            const int32_t row0 = job.m * S::kM + warp_row, row = row0 + lane;
            const int64_t col0 = static_cast<int64_t>(job.n) * NT + half * kHalf;
            bool ok;
            // next sum in TMEM, and its release once this warp has read it
            const auto wait_sum = [&] {
                ok = warp_wait(&sh->acc_full[acc], acc_phase, &sh->failed, q.dev_status);
                __syncwarp();
                tc_fence_after();
                return tmem + lanes + acc * NT + half * kHalf;
            };
            const auto sum_read = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (CTAS == 2)
                        mbar_arrive_remote(map_to_rank(smem_addr(&sh->acc_empty[acc]), 0));
                    else
                        mbar_arrive(&sh->acc_empty[acc]);
                }
                acc ^= 1;
                acc_phase ^= acc == 0 ? 1u : 0u;
            };
            // the tile's sums, segment by segment
            float sums[kChunks][32];
            const auto add_segments = [&] {
                const int32_t n_blocks = (job.k1 - job.k0) * q.pairs;
                const int32_t seg = MODE == kLinGrads ? max(n_blocks, 1) : (is_grads(MODE) ? kSegGrads : q.seg);
                for (int32_t kb = 0; kb == 0 || kb < n_blocks; kb += seg) {
                    const uint32_t src = wait_sum();
                    if (!ok)
                        return false;
#pragma unroll
                    for (int c = 0; c < kHalf; c += 16)
                        tmem_add16(src + c, &sums[c / 32][c % 32], kb == 0);
                    sum_read();
                }
                return true;
            };
            if constexpr (!is_grads(MODE)) {
                // this row's gathered columns, as bits of this half
                uint32_t hit[kChunks];
#pragma unroll
                for (int w = 0; w < kChunks; ++w)
                    hit[w] = 0;
                uint32_t hits = 0;  // dz, bit k: target k is among them
                float2 g = make_float2(0.0f, 0.0f);
                if (row < live) {
                    if (MODE == kLinDz)
                        g = q.grow[row];
                    for (int k = 0; k < q.k; ++k) {
                        const int64_t j = target_column(q, static_cast<int64_t>(row) * q.k + k, q.v0 + col0);
                        if (j >= 0 && j < kHalf) {
                            hits |= MODE == kLinDz ? 1u << k : 0u;
#pragma unroll
                            for (int w = 0; w < kChunks; ++w)
                                if (MODE == kLinStats && j >> 5 == w)
                                    hit[w] |= 1u << (j & 31);
                        }
                    }
                }
                if (!add_segments())
                    break;
                RowStats st;
#pragma unroll
                for (int ch = 0; ch < kChunks; ++ch) {
                    float(&v)[32] = sums[ch];
                    const int64_t c0 = col0 + ch * 32;
                    const int64_t end = q.vocab - (q.v0 + c0);  // columns of this chunk that exist
                    if (MODE == kLinStats) {
                        if (q.z != nullptr && row < live) {
                            float *o = q.z + row * q.z_pitch + q.v0 + c0;
#pragma unroll
                            for (int j = 0; j < 32; j += 8)
                                st_v8(o + j, v + j);
                        }
                        if (end < 32) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                v[j] = j < end ? v[j] : kNegInf;
                        }
                        const uint32_t mine = hit[ch];
                        if (mine != 0) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                v[j] = mine >> j & 1u ? kNegInf : v[j];
                        }
                        st.add(v, q.c);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            v[j] = row < live && j < end ? g.y * ex2((v[j] - g.x) * q.c) : 0.0f;
                        __nv_bfloat16 *out = q.dz + static_cast<int64_t>(row) * q.piece + c0;
                        for (int z = 0; z < q.planes; ++z, out += q.dz_plane) {
#pragma unroll
                            for (int j = 0; j < 32; j += 16) {
                                uint32_t w[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    w[i] = pack_bf16(v[j + 2 * i], v[j + 2 * i + 1]);
                                    const float2 f = bf16x2_to_float2(w[i]);
                                    v[j + 2 * i] -= f.x;
                                    v[j + 2 * i + 1] -= f.y;
                                }
                                st_v8(out + j, w);
                            }
                        }
                    }
                }
                if (MODE == kLinStats && row < live && q.v0 + col0 < q.vocab)
                    q.partials[static_cast<int64_t>(row) * q.partial_tiles + (q.v0 + col0) / kHalf] =
                        make_float2(st.s == st.s ? st.m : (st.m == kNegInf ? 0.0f : st.m), st.s);
                if (MODE == kLinDz) {
                    // the gathered columns, over what this thread wrote above
                    for (; hits != 0; hits &= hits - 1) {
                        const int64_t at = static_cast<int64_t>(row) * q.k + __ffs(hits) - 1;
                        float x = q.dzt[at];
                        __nv_bfloat16 *out = q.dz + static_cast<int64_t>(row) * q.piece + (q.tgt[at] - q.v0);
                        for (int z = 0; z < q.planes; ++z, out += q.dz_plane) {
                            const __nv_bfloat16 w = __float2bfloat16_rn(x);
                            *out = w;
                            x -= __bfloat162float(w);
                        }
                    }
                }
            } else {
                // 32 of this row's columns into dhidden's sums or dweight
                const auto put = [&](int ch, float(&v)[32]) {
                    const int64_t c0 = col0 + ch * 32;
                    if (!job.dw) {
                        if (row >= live)
                            return;
                        float *out = q.dh + (static_cast<int64_t>(job.split) * jobs.tm * S::kM + row) * q.dh_pitch + c0;
#pragma unroll
                        for (int j = 0; j < 32; j += 8)
                            if (c0 + j < q.dim) {
                                float x[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    x[i] = any ? v[j + i] : 0.0f;
                                if (!q.first) {
#pragma unroll
                                    for (int i = 0; i < 8; i += 4) {
                                        const float4 old = *reinterpret_cast<const float4 *>(out + j + i);
                                        x[i] += old.x;
                                        x[i + 1] += old.y;
                                        x[i + 2] += old.z;
                                        x[i + 3] += old.w;
                                    }
                                }
                                st_v8(out + j, x);
                            }
                        return;
                    }
                    if (q.v0 + row0 >= q.vocab || c0 >= q.dim)
                        return;
                    const int64_t at = (q.v0 + row) * q.dweight_stride + c0;
                    const bool mine = q.v0 + row < q.vocab;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[j] = any ? alpha * v[j] : 0.0f;
                    if (q.vec == 0 || c0 + 32 > q.dim) {
                        const int64_t base = (q.v0 + row0) * q.dweight_stride + c0;
                        const int32_t rows = static_cast<int32_t>(min(static_cast<int64_t>(32), q.vocab - q.v0 - row0));
                        const int32_t cols = static_cast<int32_t>(min(static_cast<int64_t>(32), q.dim - c0));
                        if (q.bf16)
                            store_rows_turned(sh->turn[warp - 2], v, static_cast<__nv_bfloat16 *>(q.dweight) + base,
                                              q.dweight_stride, rows, cols, q.accumulate != 0);
                        else
                            store_rows_turned(sh->turn[warp - 2], v, static_cast<float *>(q.dweight) + base,
                                              q.dweight_stride, rows, cols, q.accumulate != 0);
                    } else if (mine) {
                        if (q.bf16)
                            store_row(static_cast<__nv_bfloat16 *>(q.dweight) + at, v, q.accumulate != 0, q.vec == 32);
                        else
                            store_row(static_cast<float *>(q.dweight) + at, v, q.accumulate != 0, q.vec == 32);
                    }
                };
                if constexpr (MODE == kLinGrads) {
                    const uint32_t src = wait_sum();
                    if (!ok)
                        break;
#pragma unroll 1
                    for (int ch = 0; ch < kChunks; ++ch) {
                        float v[32];
                        tmem_add16(src + ch * 32, v, true);
                        tmem_add16(src + ch * 32 + 16, v + 16, true);
                        if (ch == kChunks - 1)  // the tile after next may start
                            sum_read();
                        put(ch, v);
                        // the lanes of a tile's last rows part in there, and
                        // the next loads from TMEM are the whole warp's
                        __syncwarp();
                    }
                } else {
                    if (!add_segments())
                        break;
#pragma unroll
                    for (int ch = 0; ch < kChunks; ++ch)
                        put(ch, sums[ch]);
                }
            }
        }
        if (MODE == kLinStats)
            make_dots();
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
    if (CTAS == 2)
        cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_free<CTAS>(tmem, S::kTmemCols);
    }
    if (CTAS == 2) {
        __syncthreads();
        cluster_sync();
    }
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

// Let a kernel use this much shared memory, once per kernel and device.
template <int MODE, int CTAS, int NT, typename K>
cudaError_t allow_smem(K *kernel, uint32_t bytes)
{
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t{1} << dev : 0;
    if (e != cudaSuccess || (done.load(std::memory_order_relaxed) & bit) != 0)
        return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e == cudaSuccess)
        done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

template <int MODE, int CTAS, int NT>
cudaError_t launch_mma(const CUtensorMap *maps, const MmaArgs &q, int64_t tiles, cudaStream_t s)
{
    const int sms = device_sm_count();
    if (sms < 2)
        return cudaErrorInvalidDevice;
    const auto kernel = lin_mma_kernel<MODE, CTAS, NT>;
    cudaError_t e = allow_smem<MODE, CTAS, NT>(kernel, smem_bytes<CTAS, NT>());
    if (e != cudaSuccess)
        return e;
    const int64_t units = tiles < sms / CTAS ? tiles : sms / CTAS;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(CTAS * units));
    cfg.blockDim = dim3(kMmaThreads);
    cfg.dynamicSmemBytes = smem_bytes<CTAS, NT>();
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CTAS;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CTAS == 2 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kernel, maps[0], maps[1], maps[2], maps[3], q);
    note_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int MODE>
cudaError_t launch_shape(LinTile shape, const CUtensorMap *maps, const MmaArgs &q, int64_t tiles,
                         cudaStream_t s)
{
    if (shape.ctas == 2)
        return launch_mma<MODE, 2, 256>(maps, q, tiles, s);
    if (shape.n == 256)
        return launch_mma<MODE, 1, 256>(maps, q, tiles, s);
    return shape.n == 128 ? launch_mma<MODE, 1, 128>(maps, q, tiles, s)
                          : launch_mma<MODE, 1, 64>(maps, q, tiles, s);
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
    q.v0 = v0;
    q.vocab = p.vocab;
    q.c = p.c;
    q.k = static_cast<int32_t>(p.k);
    q.tgt = p.tgt;
    q.dim = p.dim;
    q.seg = p.rows <= 128 ? kSegShort : kSegLogits;
    return q;
}

int64_t ceil_div(int64_t n, int64_t d) { return (n + d - 1) / d; }

// Rows of A's box: no more than the call has, so that a few rows cost a few.
uint32_t box_rows(const LinParams &p, LinTile shape)
{
    return shape.ctas == 1 && p.rows < 128 ? static_cast<uint32_t>(ceil_div(p.rows, 8) * 8) : 128u;
}

}  // namespace

// The tile shape with the least estimated time.  Measured at 8192 x 76032 x
// 2560 (forward): 256 x 256 by pairs 2002 TFLOP/s, 128 x 256 1697, 128 x 128
// 1271, 128 x 64 683; the last two are bound by the operands' way from L2 (24
// to 32 KB a block).  Taking pairs as 620 cycles per 64-deep block the others
// are 731, 489 and 455.  The table's 450 and 420 are those less 8% (the choice
// between the two is the same), its 680 and the 4 us (8000) that a launch of
// pairs costs more are fitted to forwards of fewer rows, pairs and 128 x 256:
// 1843 x 151936 x 2560 804 and 850 us, 2048 x 32768 x 1024 112 and 117, 1500 x
// 8192 x 1024 47 and 42, 384 x 152064 x 4096 361 and 341.  A launch's first and
// last tile add about 2000 + 10 per column that no other tile hides.
LinTile choose_tile(LinWork a, LinWork b)
{
    constexpr LinTile shapes[4] = {{2, 256}, {1, 256}, {1, 128}, {1, 64}};
    constexpr int64_t cycles[4] = {620, 680, 450, 420};
    LinTile best = shapes[0];
    int64_t least = INT64_MAX;
    for (int i = 0; i < 4; ++i) {
        const LinTile t = shapes[i];
        const int64_t units = kLinSms / t.ctas, m = 128 * t.ctas;
        int64_t cost = 2000 + 10 * t.n + (t.ctas == 2 ? 8000 : 0), longest = 0, sum = 0;
        for (const LinWork &w : {a, b}) {
            const int64_t tiles = ceil_div(w.m, m) * ceil_div(w.n, t.n);
            const int64_t depth = w.split ? ceil_div(w.depth, ceil_div(units, tiles > 0 ? tiles : 1)) : w.depth;
            sum += tiles * (w.depth * cycles[i] + 500);
            if (tiles > 0 && depth > longest)
                longest = depth;
            // whole waves where every tile is as deep
            if (b.m == 0)
                cost += ceil_div(tiles, units) * w.depth * cycles[i];
        }
        if (b.m != 0)
            cost += sum / units > longest * cycles[i] ? sum / units : longest * cycles[i];
        if (cost < least) {
            least = cost;
            best = t;
        }
    }
    return best;
}

cudaError_t lin_stats(const LinParams &p, cudaStream_t s)
{
    const int64_t step = p.weight_direct ? p.vocab : p.wpack_rows;
    const LinTile shape = p.logits_tile;
    for (int64_t v0 = 0; v0 < p.vocab; v0 += step) {
        const int64_t v1 = v0 + step < p.vocab ? v0 + step : p.vocab;
        Weight w;
        cudaError_t e = piece_weight(p, v0, v1, v0 > 0 || lin_weight_packed(p), w, s);
        CUtensorMap maps[4] = {};
        MmaArgs q = base_args(p, v0);
        q.a_rows = static_cast<int32_t>(box_rows(p, shape));
        if (p.direct) {
            q.direct_rows = static_cast<int32_t>(p.rows);
            q.targets = p.targets;
            if (e == cudaSuccess)
                e = make_map(&maps[0], p.hidden, p.dim, p.rows, p.hidden_stride, 1, p.hidden_stride, q.a_rows);
        } else if (e == cudaSuccess) {
            e = make_map(&maps[0], p.hpack, p.dim, p.rows, p.pitch, p.planes, p.hpack_plane, q.a_rows);
        }
        if (e == cudaSuccess)
            e = make_map(&maps[1], w.base, p.dim, w.rows, w.stride, p.planes, w.plane,
                         static_cast<uint32_t>(shape.n / shape.ctas));
        if (e != cudaSuccess)
            return e;
        q.blocks = static_cast<int32_t>(ceil_div(p.dim, kDepth));
        q.tiles_n = static_cast<int32_t>(ceil_div(v1 - v0, shape.n));
        q.b_row0 = static_cast<int32_t>(w.row0);
        // of the launches over parts of the table the first makes all the
        // gathered columns' logits
        q.hidden = p.hidden;
        q.weight = p.weight;
        q.hidden_stride = p.hidden_stride;
        q.weight_stride = p.weight_stride;
        q.row_list = p.row_list;
        q.xt = v0 == 0 && !lin_dots_in_pack(p) ? p.xt : nullptr;
        if (p.fused) {
            q.z = p.z;
            q.z_pitch = p.piece;
        }
        q.partials = p.partials;
        q.partial_tiles = p.tiles;
        e = launch_shape<kLinStats>(shape, maps, q, ceil_div(p.rows, 128 * shape.ctas) * q.tiles_n, s);
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

cudaError_t lin_grads(const LinParams &p, cudaStream_t s)
{
    const LinTile lt = p.logits_tile, gt = p.grads_tile;
    for (int64_t v0 = 0; v0 < p.vocab; v0 += p.piece) {
        const int64_t v1 = v0 + p.piece < p.vocab ? v0 + p.piece : p.vocab;
        Weight w;
        cudaError_t e = piece_weight(p, v0, v1, v0 > 0 || p.fused || lin_weight_packed(p), w, s);
        CUtensorMap logits[4] = {}, grads[4] = {};
        const auto map = [&e](CUtensorMap *m, const void *base, int64_t inner, int64_t rows,
                              int64_t stride, int64_t planes, int64_t plane, uint32_t box) {
            if (e == cudaSuccess)
                e = make_map(m, base, inner, rows, stride, planes, plane, box);
        };
        MmaArgs q = base_args(p, v0);
        q.a_rows = static_cast<int32_t>(box_rows(p, lt));
        map(&logits[0], p.hpack, p.dim, p.rows, p.pitch, p.planes, p.hpack_plane, q.a_rows);
        map(&logits[1], w.base, p.dim, w.rows, w.stride, p.planes, w.plane,
            static_cast<uint32_t>(lt.n / lt.ctas));
        map(&grads[0], p.dz, p.piece, p.rows_pad, p.piece, p.planes, p.dz_plane, 128);
        map(&grads[1], w.base, p.dim, w.rows, w.stride, p.planes, w.plane, 64);
        map(&grads[2], p.dz, p.piece, p.rows_pad, p.piece, p.planes, p.dz_plane, 64);
        map(&grads[3], p.hpack, p.dim, p.rows_pad, p.pitch, p.planes, p.hpack_plane, 64);
        if (e != cudaSuccess)
            return e;
        q.b_row0 = static_cast<int32_t>(w.row0);
        q.grow = p.grow;
        q.dzt = p.dzt;
        q.dz = static_cast<__nv_bfloat16 *>(p.dz);
        q.piece = p.piece;
        q.dz_plane = p.dz_plane;
        q.blocks = static_cast<int32_t>(ceil_div(p.dim, kDepth));
        q.tiles_n = static_cast<int32_t>(ceil_div(v1 - v0, lt.n));
        if (p.fused && p.z != nullptr)
            e = lin_dz(p, s);
        else
            e = launch_shape<kLinDz>(lt, logits, q, ceil_div(p.rows, 128 * lt.ctas) * q.tiles_n, s);
        if (e != cudaSuccess)
            return e;
        q.blocks = static_cast<int32_t>(ceil_div(v1 - v0, kDepth));
        q.units = device_sm_count() / gt.ctas;
        q.piece_blocks = static_cast<int32_t>(ceil_div(p.piece, kDepth));
        q.tiles_n = static_cast<int32_t>(ceil_div(p.dim, gt.n));
        const int64_t most_splits = p.dhidden != nullptr ? kMaxSplits : 0;
        if (p.dhidden != nullptr) {
            q.want_dh = 1;
            q.first = v0 == 0;
            q.dh = p.dh;
            q.dh_pitch = p.dh_pitch;
            q.dh_room = p.dh_room;
        }
        if (p.dweight != nullptr) {
            const size_t es = p.bf16 ? 2 : 4;
            q.tiles_v = static_cast<int32_t>(ceil_div(v1 - v0, 128 * gt.ctas));
            q.dweight = p.dweight;
            q.dweight_stride = p.dweight_stride;
            q.accumulate = p.accumulate;
            q.bf16 = p.bf16;
            const uintptr_t rows = reinterpret_cast<uintptr_t>(p.dweight) |
                                   static_cast<uintptr_t>(p.dweight_stride) * es;
            q.vec = rows % 32 == 0 ? 32 : (rows % 16 == 0 ? 16 : 0);
        }
        const int64_t tiles = (ceil_div(p.rows, 128 * gt.ctas) * most_splits + q.tiles_v) * q.tiles_n;
        e = p.planes == 1 ? launch_shape<kLinGrads>(gt, grads, q, tiles, s)
                          : launch_shape<kLinGradsSplit>(gt, grads, q, tiles, s);
        if (e != cudaSuccess)
            return e;
    }
    return p.dhidden == nullptr ? cudaSuccess : lin_finish(p, s);
}

}  // namespace gbce
