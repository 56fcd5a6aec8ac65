// Rows of a [vocab, dim] table by token, and the gradient of that lookup.
//
//   out[r]    = scale * table[token[r]]               (0 where the token is ignored)
//   dtable[v] (+)= scale * sum_{r : token[r] = v} grad[r]
//
// Both move rows and are bound by memory: the lookup reads and writes rows x
// dim, the gradient reads rows x dim and writes the whole table once (or,
// accumulating, reads and writes the rows that tokens name).
//
// The gradient sorts the tokens first (stable, so that a token's rows stay in
// row order and the sums are the same bits every time; no atomics), then
// walks the sorted list in chunks: a chunk sums each run of one token and
// writes the table rows whose run it holds whole; runs that cross chunks
// leave partial sums, which a last kernel joins in chunk order.  So a very
// common token is spread over many CTAs.  The zeros of rows that nobody names
// go out beside the sort or beside the chunks (see lookup_bwd).  8192 tokens,
// 152064 x 2560 bf16: 146 us where the bytes alone take 120; the sort (12 us
// of one CTA) hides behind the zeros, the named rows (20 us) come after them.
#include <cmath>
#include <cstdint>

#include "gbce_kernels.cuh"

namespace gbce {

namespace {

// ------------------------------------------------------------------ sorting

constexpr int kSortThreads = 1024, kSortWarps = 32, kSortSteps = 8;
constexpr int kSortChunk = kSortThreads * kSortSteps;  // keys a CTA takes
constexpr int kDigits = 256;
constexpr int kZeroRows = 16;  // table rows that one CTA of zeros looks after

struct SortShared {
    uint32_t count[kSortWarps][kDigits];  // then: where the warp's next key of a digit goes
    uint32_t scan[8];
};

// Token of row r as a key: its own value, or `vocab` (which sorts last) for
// one that is ignored or out of range.
__device__ __forceinline__ uint32_t token_key(const int64_t *tokens, int64_t r, int64_t vocab,
                                              int64_t ignore_index, int32_t *dev_status)
{
    const int64_t t = tokens[r];
    if (t == ignore_index)
        return static_cast<uint32_t>(vocab);
    if (t < 0 || t >= vocab) {
        report(dev_status, GBCE_DEV_BAD_INDEX);
        return static_cast<uint32_t>(vocab);
    }
    return static_cast<uint32_t>(t);
}

// Digit counts of this CTA's keys, each warp over its own run of them;
// rank[it] is the key's place among its warp's of that digit.
__device__ __forceinline__ void sort_count(SortShared &sh, const uint32_t (&key)[kSortSteps],
                                           const bool (&in)[kSortSteps], uint32_t (&rank)[kSortSteps],
                                           int shift)
{
    for (int i = threadIdx.x; i < kSortWarps * kDigits; i += kSortThreads)
        (&sh.count[0][0])[i] = 0;
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int it = 0; it < kSortSteps; ++it) {
        const uint32_t d = in[it] ? key[it] >> shift & (kDigits - 1) : kDigits;
        const unsigned same = __match_any_sync(0xffffffffu, d);
        const unsigned below = same & ((1u << lane) - 1u);
        const uint32_t had = in[it] ? sh.count[warp][d] : 0u;
        rank[it] = had + __popc(below);
        __syncwarp();
        if (in[it] && below == 0)
            sh.count[warp][d] = had + __popc(same);
        __syncwarp();
    }
    __syncthreads();
}

// Per-digit totals of the CTA to exclusive positions: count[w][d] becomes the
// place of warp w's first key of digit d.  `first` is this digit's place when
// the caller has it (several CTAs), else the digits follow one another.
__device__ __forceinline__ void sort_places(SortShared &sh, const uint32_t *first)
{
    const int d = threadIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t total = 0;
    if (d < kDigits)
        for (int w = 0; w < kSortWarps; ++w)
            total += sh.count[w][d];
    uint32_t at = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, at, o);
        at += lane >= o ? up : 0;
    }
    if (d < kDigits && lane == 31)
        sh.scan[warp] = at;
    __syncthreads();
    if (d < kDigits) {
        for (int w = 0; w < warp; ++w)
            at += sh.scan[w];
        at -= total;
        if (first != nullptr)
            at = first[d];
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t n = sh.count[w][d];
            sh.count[w][d] = at;
            at += n;
        }
    }
    __syncthreads();
}

// Index of this thread's it-th key in its CTA's chunk.
__device__ __forceinline__ int sort_slot(int it)
{
    return (threadIdx.x >> 5) * (kSortSteps * 32) + it * 32 + (threadIdx.x & 31);
}

struct SortArgs {
    const int64_t *tokens;
    int64_t n, vocab, ignore_index;
    uint32_t *keys[2], *rows[2];
    uint32_t *hist;  // [kDigits, ctas]
    int64_t ctas;
    int passes;
    int32_t *dev_status;
};

}  // namespace

// Zeros in every row of the table, kZeroRows rows to a CTA.
struct ZeroArgs {
    void *table;
    int64_t vocab, row_bytes, stride_bytes;  // row_bytes a multiple of `width`
    int width;                               // 16, 4 or 2 bytes a store
    int64_t ctas;                            // 0: nothing to write
};

// `bytes` of zeros from `at` by the CTA's threads, `width` bytes a store.
__device__ __forceinline__ void zero_bytes(char *at, int64_t bytes, int width)
{
    for (int64_t b = static_cast<int64_t>(threadIdx.x) * width; b < bytes;
         b += static_cast<int64_t>(blockDim.x) * width) {
        if (width == 16)
            *reinterpret_cast<uint4 *>(at + b) = make_uint4(0, 0, 0, 0);
        else if (width == 4)
            *reinterpret_cast<uint32_t *>(at + b) = 0;
        else
            *reinterpret_cast<uint16_t *>(at + b) = 0;
    }
}

__device__ __forceinline__ void zero_rows(const ZeroArgs &z, int64_t cta)
{
    const int64_t v0 = cta * kZeroRows, v1 = min(z.vocab, v0 + kZeroRows);
    char *first = static_cast<char *>(z.table) + v0 * z.stride_bytes;
    if (z.row_bytes == z.stride_bytes) {
        // rows without gaps are one run of bytes, which starts on 16 where the
        // table does (16 rows of 2-byte elements are 32 bytes or a multiple)
        const int64_t bytes = (v1 - v0) * z.row_bytes;
        const int64_t wide = reinterpret_cast<uintptr_t>(z.table) % 16 == 0 ? bytes / 16 * 16 : 0;
        zero_bytes(first, wide, 16);
        zero_bytes(first + wide, bytes - wide, z.width);
        return;
    }
    for (int64_t v = v0; v < v1; ++v, first += z.stride_bytes)
        zero_bytes(first, z.row_bytes, z.width);
}

// Few tokens (one chunk): every pass in one CTA, the list in shared memory,
// while the launch's other CTAs write the table's zeros.  The sorted list
// ends in buffer 0.
constexpr uint32_t kSortOneSmem = sizeof(SortShared) + 2 * kSortChunk * 4;

__global__ void __launch_bounds__(kSortThreads) embedding_sort_one(SortArgs a, ZeroArgs z)
{
    extern __shared__ uint32_t dyn[];
    grid_dependency_wait();
    launch_dependents();
    if (blockIdx.x > 0) {
        zero_rows(z, static_cast<int64_t>(blockIdx.x) - 1);
        return;
    }
    SortShared &sh = *reinterpret_cast<SortShared *>(dyn);
    uint32_t *s_key = dyn + sizeof(SortShared) / 4, *s_row = s_key + kSortChunk;
    uint32_t key[kSortSteps], row[kSortSteps], rank[kSortSteps];
    bool in[kSortSteps];
#pragma unroll
    for (int it = 0; it < kSortSteps; ++it) {
        const int i = sort_slot(it);
        in[it] = i < a.n;
        key[it] = in[it] ? token_key(a.tokens, i, a.vocab, a.ignore_index, a.dev_status) : 0u;
        row[it] = static_cast<uint32_t>(i);
    }
    for (int p = 0; p < a.passes; ++p) {
        sort_count(sh, key, in, rank, 8 * p);
        sort_places(sh, nullptr);
#pragma unroll
        for (int it = 0; it < kSortSteps; ++it)
            if (in[it]) {
                const uint32_t to = sh.count[threadIdx.x >> 5][key[it] >> (8 * p) & (kDigits - 1)] + rank[it];
                s_key[to] = key[it];
                s_row[to] = row[it];
            }
        __syncthreads();
#pragma unroll
        for (int it = 0; it < kSortSteps; ++it)
            if (in[it]) {
                key[it] = s_key[sort_slot(it)];
                row[it] = s_row[sort_slot(it)];
            }
        __syncthreads();
    }
#pragma unroll
    for (int it = 0; it < kSortSteps; ++it)
        if (in[it]) {
            a.keys[0][sort_slot(it)] = key[it];
            a.rows[0][sort_slot(it)] = row[it];
        }
}

// Many tokens: a pass is three launches.
// This CTA's keys of pass p (the first makes them from the tokens).
__device__ __forceinline__ void sort_load(const SortArgs &a, int p, uint32_t (&key)[kSortSteps],
                                          bool (&in)[kSortSteps], bool tell)
{
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kSortChunk;
#pragma unroll
    for (int it = 0; it < kSortSteps; ++it) {
        const int64_t i = base + sort_slot(it);
        in[it] = i < a.n;
        key[it] = 0u;
        if (in[it])
            key[it] = p == 0 ? token_key(a.tokens, i, a.vocab, a.ignore_index,
                                         tell ? a.dev_status : nullptr)
                             : a.keys[p & 1][i];
    }
}

__global__ void __launch_bounds__(kSortThreads) embedding_sort_count(SortArgs a, ZeroArgs z, int p)
{
    __shared__ SortShared sh;
    grid_dependency_wait();
    launch_dependents();
    if (blockIdx.x >= a.ctas) {
        zero_rows(z, static_cast<int64_t>(blockIdx.x) - a.ctas);
        return;
    }
    uint32_t key[kSortSteps], rank[kSortSteps];
    bool in[kSortSteps];
    sort_load(a, p, key, in, true);
    sort_count(sh, key, in, rank, 8 * p);
    if (threadIdx.x < kDigits) {
        uint32_t total = 0;
        for (int w = 0; w < kSortWarps; ++w)
            total += sh.count[w][threadIdx.x];
        a.hist[threadIdx.x * a.ctas + blockIdx.x] = total;
    }
}

// Exclusive sums over the [digit, cta] counts, in place (one CTA).
__global__ void __launch_bounds__(kSortThreads) embedding_sort_scan(SortArgs a, int64_t n)
{
    __shared__ uint32_t s_warp[kSortWarps];
    grid_dependency_wait();
    launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t base = 0;
    for (int64_t i0 = 0; i0 < n; i0 += kSortThreads) {
        const int64_t i = i0 + threadIdx.x;
        const uint32_t own = i < n ? a.hist[i] : 0u;
        uint32_t at = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, at, o);
            at += lane >= o ? up : 0;
        }
        if (lane == 31)
            s_warp[warp] = at;
        __syncthreads();
        uint32_t before = base, total = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            before += w < warp ? s_warp[w] : 0;
            total += s_warp[w];
        }
        if (i < n)
            a.hist[i] = before + at - own;
        base += total;
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kSortThreads) embedding_sort_scatter(SortArgs a, int p)
{
    __shared__ SortShared sh;
    __shared__ uint32_t s_first[kDigits];
    grid_dependency_wait();
    launch_dependents();
    if (threadIdx.x < kDigits)
        s_first[threadIdx.x] = a.hist[threadIdx.x * a.ctas + blockIdx.x];
    uint32_t key[kSortSteps], rank[kSortSteps];
    bool in[kSortSteps];
    sort_load(a, p, key, in, false);
    sort_count(sh, key, in, rank, 8 * p);
    sort_places(sh, s_first);
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kSortChunk;
#pragma unroll
    for (int it = 0; it < kSortSteps; ++it)
        if (in[it]) {
            const uint32_t to = sh.count[threadIdx.x >> 5][key[it] >> (8 * p) & (kDigits - 1)] + rank[it];
            const int64_t i = base + sort_slot(it);
            a.keys[(p + 1) & 1][to] = key[it];
            a.rows[(p + 1) & 1][to] = p == 0 ? static_cast<uint32_t>(i) : a.rows[p & 1][i];
        }
}

namespace {

// ------------------------------------------------------------- moving rows

// VEC elements at a time: 16 bytes, or one element where rows do not start on
// 16 bytes.
template <typename T, int VEC> struct Pack {
    __device__ static void load(const T *p, float (&f)[VEC])
    {
        if constexpr (VEC == 1) {
            f[0] = static_cast<float>(*p);
        } else {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            Elem<T>::unpack(v, f);
        }
    }
    __device__ static void store(T *p, const float (&f)[VEC])
    {
        if constexpr (VEC == 1)
            *p = T(f[0]);
        else
            *reinterpret_cast<uint4 *>(p) = Elem<T>::pack(f);
    }
};

constexpr int kMoveThreads = 128;

}  // namespace

template <typename T, int VEC>
__global__ void __launch_bounds__(256)
    embedding_lookup_kernel(const T *table, int64_t table_stride, int64_t vocab, int64_t dim,
                            const int64_t *tokens, int64_t ignore_index, float scale, T *out,
                            int64_t out_stride, int32_t *dev_status)
{
    const int64_t r = blockIdx.x;
    const int64_t t = tokens[r];
    T *dst = out + r * out_stride;
    const bool skip = t == ignore_index, bad = !skip && (t < 0 || t >= vocab);
    if (bad && threadIdx.x == 0)
        report(dev_status, GBCE_DEV_BAD_INDEX);
    const float fill = bad ? __int_as_float(0x7fc00000) : 0.0f;
    const T *src = table + (skip || bad ? 0 : t) * table_stride;
#pragma unroll 2
    for (int64_t d = static_cast<int64_t>(threadIdx.x) * VEC; d < dim; d += 256 * VEC) {
        float f[VEC];
        if (skip || bad) {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                f[i] = fill;
        } else {
            Pack<T, VEC>::load(src + d, f);
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                f[i] *= scale;
        }
        Pack<T, VEC>::store(dst + d, f);
    }
}

struct GradArgs {
    const uint32_t *keys, *rows;  // sorted
    int64_t n, vocab, dim;
    int64_t grad_stride, table_stride;
    float scale;
    int accumulate;
    int32_t chunk;       // sorted entries a CTA walks
    int32_t chunks, columns;  // chunks, and blocks of columns
    float *partial;      // [chunks, 2, dim]
};

template <typename T, int VEC>
__device__ __forceinline__ void write_sum(T *o, const float (&sum)[VEC], const GradArgs &a)
{
    float f[VEC];
    if (a.accumulate)
        Pack<T, VEC>::load(o, f);
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        f[i] = a.accumulate ? fmaf(sum[i], a.scale, f[i]) : sum[i] * a.scale;
    Pack<T, VEC>::store(o, f);
}

// Chunks of the sorted list, then (where the sort did not write them) the
// zeros of the rows that nobody names.
template <typename T, int VEC>
__global__ void __launch_bounds__(kMoveThreads)
    embedding_grad_kernel(const T *grad, T *dtable, GradArgs a)
{
    constexpr int kMaxChunk = 512;
    __shared__ uint32_t s_key[kMaxChunk + 2], s_row[kMaxChunk];
    grid_dependency_wait();
    launch_dependents();
    const int64_t walk = static_cast<int64_t>(a.chunks) * a.columns;
    if (blockIdx.x >= walk) {
        // table rows [v0, v1): those between the keys that name them are zeros
        const int64_t v0 = (static_cast<int64_t>(blockIdx.x) - walk) * kZeroRows;
        const int64_t v1 = min(a.vocab, v0 + kZeroRows);
        __shared__ uint32_t s_named;
        if (threadIdx.x < 32) {
            // first sorted entry with key >= v0: 32 probes a step
            int64_t lo = 0, hi = a.n;  // keys before lo are < v0, from hi on >= v0
            while (hi > lo) {
                const int64_t step = (hi - lo + 31) / 32;
                const int64_t at = lo + static_cast<int64_t>(threadIdx.x) * step;
                const bool less = at < hi && a.keys[at] < v0;
                const int64_t n = __popc(__ballot_sync(0xffffffffu, less));
                if (n == 0) {
                    hi = lo;
                } else {
                    const int64_t top = lo + n * step;
                    lo += (n - 1) * step + 1;
                    hi = min(hi, top);
                }
            }
            // the 32 entries from there name most CTAs' rows; where they are not
            // all (a common token's run may be as long as the list) each of 16
            // lanes looks for one row.  262144 tokens, all one, 400000 x 8 fp32:
            // 265 us (205 where they are spread), walking the run 2047; 8192
            // as in text, 4096 x 1024 fp32: 29 us and 44.
            const int64_t at = lo + threadIdx.x;
            const int64_t key = at < a.n ? a.keys[at] : a.vocab;
            uint32_t named = __reduce_or_sync(0xffffffffu, key < v1 ? 1u << (key - v0) : 0u);
            if (__all_sync(0xffffffffu, key < v1)) {
                const int64_t want = v0 + threadIdx.x;
                bool found = false;
                if (want < v1) {
                    int64_t from = lo + 32, to = a.n;  // first entry with key >= want
                    while (from < to) {
                        const int64_t mid = (from + to) / 2;
                        if (a.keys[mid] < want)
                            from = mid + 1;
                        else
                            to = mid;
                    }
                    found = from < a.n && a.keys[from] == want;
                }
                named |= __reduce_or_sync(0xffffffffu, found ? 1u << threadIdx.x : 0u);
            }
            if (threadIdx.x == 0)
                s_named = named;
        }
        __syncthreads();
        float zero[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            zero[i] = 0.0f;
        for (int64_t v = v0; v < v1; ++v) {
            if (s_named >> (v - v0) & 1u)
                continue;
            T *o = dtable + v * a.table_stride;
            for (int64_t d = static_cast<int64_t>(threadIdx.x) * VEC; d < a.dim; d += kMoveThreads * VEC)
                Pack<T, VEC>::store(o + d, zero);
        }
        return;
    }
    const int64_t c = blockIdx.x / a.columns;
    const int64_t i0 = c * a.chunk, i1 = min(a.n, i0 + a.chunk);
    const int n = static_cast<int>(i1 - i0);
    // s_key[1 ..] with the neighbours' keys on both sides
    for (int i = threadIdx.x; i < n + 2; i += kMoveThreads) {
        const int64_t at = i0 + i - 1;
        s_key[i] = at >= 0 && at < a.n ? a.keys[at] : 0xffffffffu;
        if (i < n)
            s_row[i] = a.rows[i0 + i];
    }
    __syncthreads();
    const int64_t d = (static_cast<int64_t>(blockIdx.x % a.columns) * kMoveThreads + threadIdx.x) * VEC;
    if (d >= a.dim)
        return;
    const T *src = grad + d;
    float sum[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j)
        sum[j] = 0.0f;
    constexpr int kAhead = 8;  // rows loaded before they are added
    bool begun = s_key[1] == s_key[0];  // the run began in an earlier chunk
    for (int i = 0; i < n; i += kAhead) {
        float f[kAhead][VEC];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (i + u < n && s_key[i + u + 1] < a.vocab)
                Pack<T, VEC>::load(src + static_cast<int64_t>(s_row[i + u]) * a.grad_stride, f[u]);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (i + u >= n)
                break;
            const uint32_t key = s_key[i + u + 1];
            if (key >= a.vocab)
                return;  // ignored tokens sort last
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                sum[j] += f[u][j];
            if (key == s_key[i + u + 2] && i + u + 1 < n)
                continue;
            const bool goes_on = key == s_key[i + u + 2];
            if (begun || goes_on) {
                float *o = a.partial + (c * 2 + (begun ? 0 : 1)) * a.dim + d;
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    o[j] = sum[j];
            } else {
                write_sum<T, VEC>(dtable + static_cast<int64_t>(key) * a.table_stride + d, sum, a);
            }
            begun = false;
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                sum[j] = 0.0f;
        }
    }
}

// Runs that cross chunks: the CTA of the chunk where such a run begins joins
// its partial sums, in chunk order.
template <typename T, int VEC>
__global__ void __launch_bounds__(kMoveThreads) embedding_join_kernel(T *dtable, GradArgs a)
{
    grid_dependency_wait();
    launch_dependents();
    const int64_t c = blockIdx.x / a.columns;
    const int64_t i1 = (c + 1) * a.chunk;
    if (i1 >= a.n)
        return;
    const uint32_t key = a.keys[i1 - 1];
    if (key >= a.vocab || a.keys[i1] != key)
        return;  // no run goes on past this chunk
    const int64_t i0 = c * a.chunk;
    if (a.keys[i0] == key && i0 > 0 && a.keys[i0 - 1] == key)
        return;  // it began earlier
    // the chunks that go on with it, 32 looked at a time
    int64_t last = c;
    for (bool more = true; more;) {
        const int64_t e = last + 1 + (threadIdx.x & 31);
        const unsigned on = __ballot_sync(0xffffffffu, e < a.chunks && a.keys[e * a.chunk] == key);
        const int run = __ffs(~on) - 1;
        last += run < 0 ? 32 : run;
        more = run < 0;
    }
    const int64_t d = (static_cast<int64_t>(blockIdx.x % a.columns) * kMoveThreads + threadIdx.x) * VEC;
    if (d >= a.dim)
        return;
    float sum[VEC];
    const float *p = a.partial + (c * 2 + 1) * a.dim + d;
#pragma unroll
    for (int j = 0; j < VEC; ++j)
        sum[j] = p[j];
#pragma unroll 4
    for (int64_t e = c + 1; e <= last; ++e) {
        const float *q = a.partial + e * 2 * a.dim + d;
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            sum[j] += q[j];
    }
    write_sum<T, VEC>(dtable + static_cast<int64_t>(key) * a.table_stride + d, sum, a);
}

}  // namespace gbce

namespace {

size_t elem_size(gbce_dtype dt) { return dt == GBCE_BF16 ? 2 : 4; }

constexpr int64_t kMaxVocab = INT32_MAX - 64, kMaxDim = int64_t{1} << 20;

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
        dim > kMaxDim || !std::isfinite(scale))
        return GBCE_EINVAL;
    return GBCE_OK;
}

// Rows of both matrices start on 16 bytes and dim is whole 16-byte vectors.
bool vectors(const void *x, int64_t xs, const void *y, int64_t ys, int64_t dim, gbce_dtype dt)
{
    const uintptr_t all = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y) |
                          static_cast<uintptr_t>(xs * static_cast<int64_t>(elem_size(dt))) |
                          static_cast<uintptr_t>(ys * static_cast<int64_t>(elem_size(dt))) |
                          static_cast<uintptr_t>(dim * static_cast<int64_t>(elem_size(dt)));
    return all % 16 == 0;
}

template <typename... Args>
cudaError_t launch_after(void (*kernel)(Args...), int64_t grid, int block, size_t smem,
                         cudaStream_t s, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.dynamicSmemBytes = smem;
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(block));
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    gbce::note_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t lookup(const void *table, int64_t ts, int64_t vocab, int64_t dim, const int64_t *tokens,
                   int64_t rows, int64_t ignore_index, float scale, void *out, int64_t os,
                   int32_t *dev_status, cudaStream_t s)
{
    gbce::embedding_lookup_kernel<T, VEC><<<static_cast<unsigned>(rows), 256, 0, s>>>(
        static_cast<const T *>(table), ts, vocab, dim, tokens, ignore_index, scale,
        static_cast<T *>(out), os, dev_status);
    gbce::note_launches(1);
    return cudaGetLastError();
}

// Where the sorted list and the partial sums lie in the workspace.
struct Layout {
    size_t keys[2], rows[2], hist, partial, total;
    int64_t ctas, chunk, chunks;
};

Layout layout(int64_t n, int64_t dim)
{
    Layout w{};
    size_t off = 0;
    const auto take = [&off](int64_t count) {
        const size_t at = off;
        off += (static_cast<size_t>(count) * 4 + 255) / 256 * 256;
        return at;
    };
    w.ctas = (n + gbce::kSortChunk - 1) / gbce::kSortChunk;
    // enough chunks to spread a long list over the SMs, few enough to join
    w.chunk = n / 1024 / 32 * 32;
    w.chunk = w.chunk < 32 ? 32 : (w.chunk > 512 ? 512 : w.chunk);
    w.chunks = (n + w.chunk - 1) / w.chunk;
    for (int i = 0; i < 2; ++i) {
        w.keys[i] = take(n);
        w.rows[i] = take(n);
    }
    w.hist = take(gbce::kDigits * w.ctas);
    w.partial = take(w.chunks * 2 * dim);
    w.total = off;
    return w;
}

template <typename T, int VEC>
cudaError_t lookup_bwd(const void *grad, int64_t gs, int64_t rows, int64_t vocab, int64_t dim,
                       const int64_t *tokens, int64_t ignore_index, float scale, void *dtable,
                       int64_t ds, int accumulate, void *ws, int32_t *dev_status, cudaStream_t s)
{
    const Layout w = layout(rows, dim);
    const auto at = [ws](size_t off) { return reinterpret_cast<uint32_t *>(static_cast<char *>(ws) + off); };
    gbce::SortArgs a{};
    a.tokens = tokens;
    a.n = rows;
    a.vocab = vocab;
    a.ignore_index = ignore_index;
    for (int i = 0; i < 2; ++i) {
        a.keys[i] = at(w.keys[i]);
        a.rows[i] = at(w.rows[i]);
    }
    a.hist = at(w.hist);
    a.dev_status = dev_status;
    a.passes = 1;
    while (vocab >> (8 * a.passes) != 0)  // the keys go up to vocab itself
        ++a.passes;
    a.ctas = w.ctas;
    // Few tokens for the table's rows: the zeros of all rows go out beside the
    // sort, which leaves the memory idle, and the rows that tokens name are
    // written again (8192 tokens, 152064 x 2560 bf16: 146 us; with every zero
    // beside the chunks, where it takes a search to know who is named, 154 us).
    // Many: few zeros are left, and the chunks' launch writes just those.
    gbce::ZeroArgs z{};
    const int64_t zero_ctas = accumulate ? 0 : (vocab + gbce::kZeroRows - 1) / gbce::kZeroRows;
    if (zero_ctas > 0 && w.ctas > 0 && 2 * rows < vocab) {
        z.table = dtable;
        z.vocab = vocab;
        z.row_bytes = dim * static_cast<int64_t>(sizeof(T));
        z.stride_bytes = ds * static_cast<int64_t>(sizeof(T));
        z.width = VEC > 1 ? 16 : static_cast<int>(sizeof(T));
        z.ctas = zero_ctas;
    }
    cudaError_t e = cudaSuccess;
    if (w.ctas == 1) {
        e = cudaFuncSetAttribute(gbce::embedding_sort_one, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 gbce::kSortOneSmem);
        if (e == cudaSuccess)
            e = launch_after(gbce::embedding_sort_one, 1 + z.ctas, gbce::kSortThreads,
                             gbce::kSortOneSmem, s, a, z);
    } else if (w.ctas > 1) {
        for (int p = 0; e == cudaSuccess && p < a.passes; ++p) {
            e = launch_after(gbce::embedding_sort_count, w.ctas + (p == 0 ? z.ctas : 0),
                             gbce::kSortThreads, 0, s, a, z, p);
            if (e == cudaSuccess)
                e = launch_after(gbce::embedding_sort_scan, 1, gbce::kSortThreads, 0, s, a,
                                 gbce::kDigits * w.ctas);
            if (e == cudaSuccess)
                e = launch_after(gbce::embedding_sort_scatter, w.ctas, gbce::kSortThreads, 0, s, a, p);
        }
    }
    const int last = w.ctas > 1 ? a.passes & 1 : 0;
    gbce::GradArgs g{};
    g.keys = a.keys[last];
    g.rows = a.rows[last];
    g.n = rows;
    g.vocab = vocab;
    g.dim = dim;
    g.grad_stride = gs;
    g.table_stride = ds;
    g.scale = scale;
    g.accumulate = accumulate;
    g.chunk = static_cast<int32_t>(w.chunk);
    g.chunks = static_cast<int32_t>(w.chunks);
    g.columns = static_cast<int32_t>((dim + gbce::kMoveThreads * VEC - 1) / (gbce::kMoveThreads * VEC));
    g.partial = reinterpret_cast<float *>(at(w.partial));
    const int64_t walk = static_cast<int64_t>(g.chunks) * g.columns;
    const int64_t zeros = zero_ctas - z.ctas;
    if (e == cudaSuccess && walk + zeros > 0)
        e = launch_after(gbce::embedding_grad_kernel<T, VEC>, walk + zeros, gbce::kMoveThreads, 0, s,
                         static_cast<const T *>(grad), static_cast<T *>(dtable), g);
    if (e == cudaSuccess && g.chunks > 1)
        e = launch_after(gbce::embedding_join_kernel<T, VEC>, walk, gbce::kMoveThreads, 0, s,
                         static_cast<T *>(dtable), g);
    return e;
}

}  // namespace

extern "C" {

size_t gbce_embedding_workspace_size(int64_t rows, int64_t vocab, int64_t dim)
{
    return rows > 0 && rows <= INT32_MAX / 2 && vocab > 0 && dim > 0 && dim <= kMaxDim
               ? layout(rows, dim).total
               : 0;
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
    const bool vec = vectors(table, table_row_stride, out, out_row_stride, dim, dtype);
    const auto run = dtype == GBCE_BF16 ? (vec ? lookup<__nv_bfloat16, 8> : lookup<__nv_bfloat16, 1>)
                                        : (vec ? lookup<float, 4> : lookup<float, 1>);
    const cudaError_t e = run(table, table_row_stride, vocab, dim, tokens, rows, ignore_index, scale,
                              out, out_row_stride, dev_status, static_cast<cudaStream_t>(stream));
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
    const bool vec = vectors(rows > 0 ? grad_out : nullptr, rows > 0 ? grad_row_stride : 0, dtable,
                             dtable_row_stride, dim, dtype);
    const auto run = dtype == GBCE_BF16
                         ? (vec ? lookup_bwd<__nv_bfloat16, 8> : lookup_bwd<__nv_bfloat16, 1>)
                         : (vec ? lookup_bwd<float, 4> : lookup_bwd<float, 1>);
    const cudaError_t e = run(grad_out, grad_row_stride, rows, vocab, dim, tokens, ignore_index, scale,
                              dtable, dtable_row_stride, accumulate, workspace, dev_status,
                              static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GBCE_OK : GBCE_ECUDA;
}

}  // extern "C"
