// C-ABI entry points of the calls that start from hidden states (declared in
// include/gbce.h): host-side argument checks, workspace layout, dispatch.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/gbce.h"
#include "gbce_internal.h"
#include "gbce_linear.h"

using gbce::LinParams;

namespace {

constexpr int64_t kMaxVocab = INT32_MAX - 64;
constexpr int64_t kMaxRows = int64_t{1} << 24;
constexpr int64_t kMaxDim = int64_t{1} << 20;
// Bytes that one piece's dz, or a piece of an fp32 weight, may take beyond the
// smallest width (kLinPieceUnit columns).
constexpr int64_t kPieceBytes = int64_t{512} << 20;
// The same for a bf16 weight that has to be packed; most are read in place
// and leave this room unused.
constexpr int64_t kWeightBytes = int64_t{128} << 20;

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
size_t elem_size(gbce_dtype dt) { return dt == GBCE_BF16 ? 2 : 4; }

struct Layout {
    size_t head, row_list, row_map, tgt, xt, partials, loss, grow, dzt, hpack, wpack, z,
        dz, dh;
    size_t total;
    int64_t rows_pad, tiles, piece, pitch, wpack_rows, dh_pitch, dh_room;
    int planes;
    bool keep;
    gbce::LinTile logits_tile, grads_tile;
};

// Bytes of fp32 logits that a fused call keeps rather than forming them twice.
// Measured, formed twice -> kept: 64 x 4096 x 256 fp32 48 -> 43 us, 1922 rows
// (256 labelled) x 4096 x 1024 bf16 60 -> 51, 613 x 40001 x 1001 bf16 304 ->
// 292, 1024 x 32768 x 1024 fp32 1020 -> 816.  Beyond this size the memory is
// what the caller came to save.
constexpr int64_t kKeepBytes = int64_t{256} << 20;

// fp32 values that split sums of dhidden may take beyond one part.
constexpr int64_t kSplitRoom = int64_t{32} << 20;

// Where everything lies in the workspace.  With `backward`, the buffers of
// the gradient (and of the statistics, which a fused call needs too).
// `direct`: the weight is read in place; no layout is larger than a direct
// one's, whatever the weight's alignment.
Layout layout(int64_t rows, int64_t vocab, int64_t dim, int64_t k, gbce_dtype dt, bool backward,
              bool direct)
{
    Layout w{};
    size_t off = 0;
    const auto take = [&off](int64_t n, size_t bytes) {
        const size_t at = off;
        off += align_up(static_cast<size_t>(n) * bytes, 256);
        return at;
    };
    w.rows_pad = round_up(rows, gbce::kLinRowPad);
    const int64_t products = dt == GBCE_BF16 ? 1 : 6;
    const int64_t depth = (dim + 63) / 64 * products;
    w.logits_tile = gbce::choose_tile({rows, vocab, depth, false}, {0, 0, 0, false});
    // two halves of a tile leave their own (max, sum)
    const int64_t half = w.logits_tile.n / 2;
    w.tiles = (vocab + half - 1) / half;
    w.head = take(1, sizeof(gbce::LinHeader));
    w.row_list = take(rows, 4);
    w.row_map = take(rows, 4);
    w.tgt = take(w.rows_pad * k, 4);
    w.xt = take(w.rows_pad * k, 4);
    w.loss = take(rows, 4);
    // bf16 planes, rows on 16 bytes as the tensor maps want them
    w.planes = dt == GBCE_BF16 ? 1 : 3;
    w.pitch = round_up(dim, 8);
    w.hpack = take(w.planes * w.rows_pad * w.pitch, 2);
    const int64_t full = round_up(vocab, 256);
    int64_t wunits = (dt == GBCE_BF16 ? kWeightBytes : kPieceBytes) / (w.planes * w.pitch * gbce::kLinPieceUnit * 2);
    wunits = wunits < 1 ? 1 : wunits;
    w.wpack_rows = wunits * gbce::kLinPieceUnit < full ? wunits * gbce::kLinPieceUnit : full;
    w.wpack = take(w.planes * w.wpack_rows * w.pitch, 2);
    w.partials = take(w.rows_pad * w.tiles, 8);
    if (backward) {
        w.grow = take(w.rows_pad, 8);
        w.dzt = take(w.rows_pad * k, 4);
        // pieces of the vocabulary: whole units, as many as kPieceBytes of dz
        // allow, and no more than the packed part of the weight holds
        int64_t units = kPieceBytes / (w.planes * w.rows_pad * gbce::kLinPieceUnit * 2);
        units = units < 1 ? 1 : units;
        if (!direct && units > wunits)
            units = wunits;
        w.piece = units * gbce::kLinPieceUnit < full ? units * gbce::kLinPieceUnit : full;
        // a call whose logits are few keeps them from the statistics to the
        // gradient (fused calls)
        w.keep = w.piece >= vocab && w.rows_pad * w.piece * 4 <= kKeepBytes;
        w.z = w.keep ? take(w.rows_pad * w.piece, 4) : 0;
        w.dz = take(w.planes * w.rows_pad * w.piece, 2);
        const int64_t piece_depth = w.piece / 64 * products, row_depth = (rows + 63) / 64 * products;
        w.grads_tile = gbce::choose_tile({rows, dim, piece_depth, true}, {w.piece, dim, row_depth, false});
        w.dh_pitch = round_up(dim, 8);
        const int64_t one = w.rows_pad * w.dh_pitch;
        const int64_t most = one * gbce::kMaxSplits < kSplitRoom ? one * gbce::kMaxSplits : kSplitRoom;
        w.dh_room = one > most ? one : most;
        w.dh = take(w.dh_room, 4);
    }
    w.total = off;
    return w;
}

bool overlap(const void *a, size_t an, const void *b, size_t bn)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return an > 0 && bn > 0 && x < y + bn && y < x + an;
}

size_t span(int64_t rows, int64_t stride, int64_t dim, gbce_dtype dt)
{
    return rows == 0 ? 0 : static_cast<size_t>((rows - 1) * stride + dim) * elem_size(dt);
}

// A [n, dim] matrix of rows `stride` apart: addressable and of its type's
// alignment.  One without rows has any address; null is no matrix at all.
gbce_status check_matrix(const void *p, int64_t n, int64_t stride, int64_t dim, gbce_dtype dt)
{
    if (p == nullptr || stride < dim || stride > (INT64_MAX / 16) / (n > 0 ? n : 1))
        return GBCE_EINVAL;
    return reinterpret_cast<uintptr_t>(p) % elem_size(dt) == 0 ? GBCE_OK : GBCE_EDTYPE;
}

struct Shape {
    const void *hidden;
    int64_t hidden_stride;
    const void *weight;
    int64_t weight_stride;
    gbce_dtype dtype;
    int64_t rows, vocab, dim, k;
    float temperature;
};

// The tensor maps read bf16 rows that start on 16 bytes.
bool weight_direct(const Shape &a)
{
    return a.dtype == GBCE_BF16 && reinterpret_cast<uintptr_t>(a.weight) % 16 == 0 &&
           a.weight_stride % 8 == 0;
}

gbce_status check_shape(const Shape &a)
{
    if (a.dtype != GBCE_F32 && a.dtype != GBCE_BF16)
        return GBCE_EDTYPE;
    if (a.rows < 0 || a.rows > kMaxRows || a.vocab < 1 || a.vocab > kMaxVocab || a.dim < 1 ||
        a.dim > kMaxDim || a.k < 1 || a.k > GBCE_MAX_K || a.hidden_stride < a.dim ||
        a.weight_stride < a.dim)
        return GBCE_EINVAL;
    if (!(std::isfinite(a.temperature) && a.temperature > 0.0f))
        return GBCE_EINVAL;
    if (a.rows == 0)
        return GBCE_OK;
    const gbce_status st = check_matrix(a.hidden, a.rows, a.hidden_stride, a.dim, a.dtype);
    return st != GBCE_OK ? st : check_matrix(a.weight, a.vocab, a.weight_stride, a.dim, a.dtype);
}

struct Grads {
    void *dhidden;
    int64_t dhidden_stride;
    void *dweight;
    int64_t dweight_stride;
    bool accumulate;
};

gbce_status check_grads(const Shape &a, const Grads &g)
{
    if (g.dhidden == nullptr && g.dweight == nullptr)
        return GBCE_EINVAL;
    const size_t hb = span(a.rows, a.hidden_stride, a.dim, a.dtype);
    const size_t wb = span(a.vocab, a.weight_stride, a.dim, a.dtype);
    size_t db = 0;
    if (g.dhidden != nullptr) {
        const gbce_status st = check_matrix(g.dhidden, a.rows, g.dhidden_stride, a.dim, a.dtype);
        if (st != GBCE_OK)
            return st;
        db = span(a.rows, g.dhidden_stride, a.dim, a.dtype);
        if (overlap(g.dhidden, db, a.hidden, hb) || overlap(g.dhidden, db, a.weight, wb))
            return GBCE_EINVAL;
    }
    if (g.dweight != nullptr) {
        const gbce_status st = check_matrix(g.dweight, a.vocab, g.dweight_stride, a.dim, a.dtype);
        if (st != GBCE_OK)
            return st;
        const size_t n = span(a.vocab, g.dweight_stride, a.dim, a.dtype);
        if (overlap(g.dweight, n, a.hidden, hb) || overlap(g.dweight, n, a.weight, wb) ||
            (g.dhidden != nullptr && overlap(g.dweight, n, g.dhidden, db)))
            return GBCE_EINVAL;
    }
    return GBCE_OK;
}

gbce_status check_workspace(const void *ws, size_t bytes, const Layout &w)
{
    // tiles are stored 32 bytes at a time
    if (ws == nullptr || bytes < w.total || reinterpret_cast<uintptr_t>(ws) % 32 != 0)
        return GBCE_EWORKSPACE;
    return GBCE_OK;
}

template <typename P>
P *at(void *ws, size_t off)
{
    return reinterpret_cast<P *>(static_cast<char *>(ws) + off);
}

LinParams params(const Shape &a, const Layout &w, void *ws, bool backward, int32_t *dev_status)
{
    LinParams p{};
    p.hidden = a.hidden;
    p.weight = a.weight;
    p.hidden_stride = a.hidden_stride;
    p.weight_stride = a.weight_stride;
    p.rows = a.rows;
    p.vocab = a.vocab;
    p.dim = a.dim;
    p.bf16 = a.dtype == GBCE_BF16;
    p.k = a.k;
    p.T = a.temperature;
    p.c = static_cast<float>(1.4426950408889634 / static_cast<double>(a.temperature));
    p.head = at<gbce::LinHeader>(ws, w.head);
    p.row_list = at<int32_t>(ws, w.row_list);
    p.row_map = at<int32_t>(ws, w.row_map);
    p.tgt = at<int32_t>(ws, w.tgt);
    p.xt = at<float>(ws, w.xt);
    p.partials = at<float2>(ws, w.partials);
    p.planes = w.planes;
    p.pitch = w.pitch;
    p.hpack = at<void>(ws, w.hpack);
    p.hpack_plane = w.rows_pad * w.pitch;
    p.weight_direct = weight_direct(a);
    p.wpack = at<void>(ws, w.wpack);
    p.wpack_rows = w.wpack_rows;
    if (backward) {
        p.grow = at<float2>(ws, w.grow);
        p.dzt = at<float>(ws, w.dzt);
        p.z = w.keep ? at<float>(ws, w.z) : nullptr;
        p.dz = at<void>(ws, w.dz);
        p.dz_plane = w.rows_pad * w.piece;
        p.dh = at<float>(ws, w.dh);
        p.dh_pitch = w.dh_pitch;
        p.dh_room = w.dh_room;
    }
    p.rows_pad = w.rows_pad;
    p.tiles = w.tiles;
    p.backward = backward;
    // a forward of one row tile: nothing to gain from leaving rows out, so
    // hidden states that the tensor maps can read are read in place
    p.direct = !backward && a.rows <= 128 && a.dtype == GBCE_BF16 &&
               reinterpret_cast<uintptr_t>(a.hidden) % 16 == 0 && a.hidden_stride % 8 == 0;
    p.logits_tile = w.logits_tile;
    p.grads_tile = w.grads_tile;
    p.piece = w.piece;
    const int64_t m = 128 * w.logits_tile.ctas, n = w.logits_tile.n;
    const int64_t columns = p.weight_direct || w.wpack_rows > a.vocab ? a.vocab : w.wpack_rows;
    const int64_t tiles = (a.rows + m - 1) / m * ((columns + n - 1) / n), units = gbce::kLinSms / w.logits_tile.ctas;
    p.stats_warps = 8 * w.logits_tile.ctas * (tiles < units ? tiles : units);
    p.dev_status = dev_status;
    return p;
}

void set_grads(LinParams &p, const Grads &g)
{
    p.dhidden = g.dhidden;
    p.dweight = g.dweight;
    p.dhidden_stride = g.dhidden_stride;
    p.dweight_stride = g.dweight_stride;
    p.accumulate = g.accumulate;
}

cudaError_t forward(const LinParams &p, cudaStream_t s)
{
    const cudaError_t e = gbce::lin_stats(p, s);
    return e != cudaSuccess ? e : gbce::lin_combine(p, s);
}

bool valid_reduction(gbce_reduction r) { return r == GBCE_NONE || r == GBCE_SUM || r == GBCE_MEAN; }

gbce_status cuda_status(cudaError_t e) { return e == cudaSuccess ? GBCE_OK : GBCE_ECUDA; }

// The gradients of a call without rows: zeros in dweight, unless it
// accumulates.  What is written, and next to what, is checked as in any call.
gbce_status no_rows(const Shape &a, const Grads &g, cudaStream_t s)
{
    gbce_status st = check_matrix(a.weight, a.vocab, a.weight_stride, a.dim, a.dtype);
    if (st != GBCE_OK || (st = check_grads(a, g)) != GBCE_OK)
        return st;
    if (g.dweight == nullptr || g.accumulate)
        return GBCE_OK;
    const size_t es = elem_size(a.dtype);
    return cuda_status(cudaMemset2DAsync(g.dweight, static_cast<size_t>(g.dweight_stride) * es, 0,
                                         static_cast<size_t>(a.dim) * es, static_cast<size_t>(a.vocab), s));
}

// The loss, and with `g` both gradients after it.
gbce_status ce_call(const Shape &a, const int64_t *labels, int64_t ignore_index,
                    gbce_reduction reduction, const float *grad_out, float *loss_out,
                    float *logp_out, float *row_state_out, int64_t *n_items_out, const Grads *g,
                    void *workspace, size_t workspace_bytes, int32_t *dev_status, cudaStream_t s)
{
    gbce_status st = check_shape(a);
    if (st != GBCE_OK)
        return st;
    if (!valid_reduction(reduction))
        return GBCE_EINVAL;
    if (a.rows == 0) {
        if (reduction != GBCE_NONE && loss_out == nullptr)
            return GBCE_EINVAL;
        if (g != nullptr && (st = no_rows(a, *g, s)) != GBCE_OK)
            return st;
        cudaError_t e = cudaSuccess;
        if (reduction != GBCE_NONE)
            e = cudaMemsetAsync(loss_out, 0, sizeof(float), s);
        if (e == cudaSuccess && n_items_out != nullptr)
            e = cudaMemsetAsync(n_items_out, 0, sizeof(int64_t), s);
        return cuda_status(e);
    }
    if (labels == nullptr || loss_out == nullptr)
        return GBCE_EINVAL;
    if (g != nullptr && (st = check_grads(a, *g)) != GBCE_OK)
        return st;
    const Layout w = layout(a.rows, a.vocab, a.dim, 1, a.dtype, g != nullptr, weight_direct(a));
    if ((st = check_workspace(workspace, workspace_bytes, w)) != GBCE_OK)
        return st;
    LinParams p = params(a, w, workspace, g != nullptr, dev_status);
    p.targets = labels;
    p.token_ce = true;
    p.ignore_index = ignore_index;
    p.reduction = static_cast<int>(reduction);
    p.n_items_out = n_items_out;
    p.loss_rows = reduction == GBCE_NONE ? loss_out : at<float>(workspace, w.loss);
    p.loss_out = reduction == GBCE_NONE ? nullptr : loss_out;
    p.logp_out = logp_out;
    p.state_out = row_state_out;
    if (g != nullptr) {
        p.fused = true;
        p.grad_out = grad_out;
        set_grads(p, *g);
    }
    cudaError_t e = gbce::lin_select(p, s);
    if (e == cudaSuccess)
        e = forward(p, s);
    if (e != cudaSuccess || g == nullptr)
        return cuda_status(e);
    return cuda_status(gbce::lin_grads(p, s));
}

}  // namespace

extern "C" {

size_t gbce_linear_workspace_size(int64_t rows, int64_t vocab, int64_t dim, int64_t k,
                                  gbce_dtype dtype, int backward)
{
    if ((dtype != GBCE_F32 && dtype != GBCE_BF16) || rows <= 0 || rows > kMaxRows || vocab < 1 ||
        vocab > kMaxVocab || dim < 1 || dim > kMaxDim || k < 1 || k > GBCE_MAX_K)
        return 0;
    return layout(rows, vocab, dim, k, dtype, backward != 0, dtype == GBCE_BF16).total;
}

gbce_status linear_selective_logsoftmax(const void *hidden, int64_t hidden_row_stride,
                                        const void *weight, int64_t weight_row_stride,
                                        gbce_dtype dtype, int64_t rows, int64_t vocab, int64_t dim,
                                        const int64_t *index, int64_t k, float temperature,
                                        const uint8_t *row_mask, float *logp_out,
                                        float *row_state_out, void *workspace,
                                        size_t workspace_bytes, int32_t *dev_status, void *stream)
{
    const Shape a{hidden, hidden_row_stride, weight, weight_row_stride, dtype,
                  rows,   vocab,             dim,    k,                 temperature};
    gbce_status st = check_shape(a);
    if (st != GBCE_OK || rows == 0)
        return st;
    if (index == nullptr || logp_out == nullptr)
        return GBCE_EINVAL;
    const Layout w = layout(rows, vocab, dim, k, dtype, false, weight_direct(a));
    if ((st = check_workspace(workspace, workspace_bytes, w)) != GBCE_OK)
        return st;
    LinParams p = params(a, w, workspace, false, dev_status);
    p.targets = index;
    p.row_mask = row_mask;
    p.logp_out = logp_out;
    p.state_out = row_state_out;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = gbce::lin_select(p, s);
    if (e == cudaSuccess)
        e = forward(p, s);
    return cuda_status(e);
}

gbce_status linear_selective_logsoftmax_bwd(
    const void *hidden, int64_t hidden_row_stride, const void *weight, int64_t weight_row_stride,
    gbce_dtype dtype, int64_t rows, int64_t vocab, int64_t dim, const int64_t *index, int64_t k,
    float temperature, const uint8_t *row_mask, const float *grad_logp, const float *saved_logp,
    const float *row_state, void *dhidden, int64_t dhidden_row_stride, void *dweight,
    int64_t dweight_row_stride, int accumulate, void *workspace, size_t workspace_bytes,
    int32_t *dev_status, void *stream)
{
    const Shape a{hidden, hidden_row_stride, weight, weight_row_stride, dtype,
                  rows,   vocab,             dim,    k,                 temperature};
    const Grads g{dhidden, dhidden_row_stride, dweight, dweight_row_stride, accumulate != 0};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    gbce_status st = check_shape(a);
    if (st != GBCE_OK)
        return st;
    if (rows == 0)
        return no_rows(a, g, s);
    if (index == nullptr || grad_logp == nullptr || saved_logp == nullptr || row_state == nullptr)
        return GBCE_EINVAL;
    if ((st = check_grads(a, g)) != GBCE_OK)
        return st;
    const Layout w = layout(rows, vocab, dim, k, dtype, true, weight_direct(a));
    if ((st = check_workspace(workspace, workspace_bytes, w)) != GBCE_OK)
        return st;
    LinParams p = params(a, w, workspace, true, dev_status);
    p.targets = index;
    p.whole_rows = true;
    p.row_mask = row_mask;
    p.grad_out = grad_logp;
    p.saved_logp = saved_logp;
    p.saved_state = row_state;
    set_grads(p, g);
    cudaError_t e = gbce::lin_select(p, s);
    if (e == cudaSuccess)
        e = gbce::lin_grads(p, s);
    return cuda_status(e);
}

gbce_status linear_ce_fwd(const void *hidden, int64_t hidden_row_stride, const void *weight,
                          int64_t weight_row_stride, gbce_dtype dtype, int64_t rows, int64_t vocab,
                          int64_t dim, const int64_t *labels, int64_t ignore_index,
                          float temperature, gbce_reduction reduction, float *loss_out,
                          float *logp_out, float *row_state_out, int64_t *n_items_out,
                          void *workspace, size_t workspace_bytes, int32_t *dev_status,
                          void *stream)
{
    const Shape a{hidden, hidden_row_stride, weight, weight_row_stride, dtype,
                  rows,   vocab,             dim,    1,                 temperature};
    return ce_call(a, labels, ignore_index, reduction, nullptr, loss_out, logp_out, row_state_out,
                   n_items_out, nullptr, workspace, workspace_bytes, dev_status,
                   static_cast<cudaStream_t>(stream));
}

gbce_status linear_ce_bwd(const void *hidden, int64_t hidden_row_stride, const void *weight,
                          int64_t weight_row_stride, gbce_dtype dtype, int64_t rows, int64_t vocab,
                          int64_t dim, const int64_t *labels, int64_t ignore_index,
                          float temperature, gbce_reduction reduction, const float *grad_out,
                          const float *saved_logp, const float *row_state, const int64_t *n_items,
                          void *dhidden, int64_t dhidden_row_stride, void *dweight,
                          int64_t dweight_row_stride, int accumulate, void *workspace,
                          size_t workspace_bytes, int32_t *dev_status, void *stream)
{
    const Shape a{hidden, hidden_row_stride, weight, weight_row_stride, dtype,
                  rows,   vocab,             dim,    1,                 temperature};
    const Grads g{dhidden, dhidden_row_stride, dweight, dweight_row_stride, accumulate != 0};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    gbce_status st = check_shape(a);
    if (st != GBCE_OK)
        return st;
    if (!valid_reduction(reduction))
        return GBCE_EINVAL;
    if (rows == 0)
        return no_rows(a, g, s);
    if (labels == nullptr || grad_out == nullptr || saved_logp == nullptr || row_state == nullptr ||
        (reduction == GBCE_MEAN && n_items == nullptr))
        return GBCE_EINVAL;
    if ((st = check_grads(a, g)) != GBCE_OK)
        return st;
    const Layout w = layout(rows, vocab, dim, 1, dtype, true, weight_direct(a));
    if ((st = check_workspace(workspace, workspace_bytes, w)) != GBCE_OK)
        return st;
    LinParams p = params(a, w, workspace, true, dev_status);
    p.targets = labels;
    p.token_ce = true;
    p.ignore_index = ignore_index;
    p.grad_out = grad_out;
    p.reduction = static_cast<int>(reduction);
    p.n_items = n_items;
    p.saved_logp = saved_logp;
    p.saved_state = row_state;
    set_grads(p, g);
    cudaError_t e = gbce::lin_select(p, s);
    if (e == cudaSuccess)
        e = gbce::lin_grads(p, s);
    return cuda_status(e);
}

gbce_status linear_ce_fwd_bwd_fused(
    const void *hidden, int64_t hidden_row_stride, const void *weight, int64_t weight_row_stride,
    gbce_dtype dtype, int64_t rows, int64_t vocab, int64_t dim, const int64_t *labels,
    int64_t ignore_index, float temperature, gbce_reduction reduction, const float *grad_out,
    float *loss_out, float *logp_out, float *row_state_out, int64_t *n_items_out, void *dhidden,
    int64_t dhidden_row_stride, void *dweight, int64_t dweight_row_stride, int accumulate,
    void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream)
{
    const Shape a{hidden, hidden_row_stride, weight, weight_row_stride, dtype,
                  rows,   vocab,             dim,    1,                 temperature};
    const Grads g{dhidden, dhidden_row_stride, dweight, dweight_row_stride, accumulate != 0};
    if (rows > 0 && grad_out == nullptr)
        return GBCE_EINVAL;
    return ce_call(a, labels, ignore_index, reduction, grad_out, loss_out, logp_out, row_state_out,
                   n_items_out, &g, workspace, workspace_bytes, dev_status,
                   static_cast<cudaStream_t>(stream));
}

}  // extern "C"
