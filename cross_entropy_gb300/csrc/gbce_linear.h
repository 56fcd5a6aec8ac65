// Internal interface of the calls that start from hidden states: the logits
// are tiles of hidden . weight^T that never reach memory as a whole.
//
//   z[i, v]  = sum_d hidden[i, d] weight[v, d]
//   stats    = per (row, vocabulary tile): max and sum of exp over the columns
//              that the row does not gather, and its gathered columns' logits
//   dz[i, v] = coef_i 2^{(z - M_i) c} / S_i, gathered columns in the expm1 form
//   dhidden  = alpha dz . weight          dweight = alpha dz^T . hidden
//
// Rows that take no part (masked, ignored, or with a label out of range) are
// left out first: the kernels work on the live rows, packed one after another.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gbce {

// Rows of the packed buffers are padded to this many, columns of a piece to
// as many.
constexpr int kLinRowPad = 256;
// The GPU's SMs, for choices that the workspace's layout depends on (a pure
// function of a call's sizes).
constexpr int64_t kLinSms = 152;
// Vocabulary columns in one piece of the backward: a multiple of this, a
// 256-wide tile for each pair of SMs.
constexpr int64_t kLinPieceUnit = kLinSms / 2 * 256;
// The most parts that dhidden's sums over a piece are split into.
constexpr uint32_t kMaxSplits = 64;

// A tile shape of the products: 128 rows per CTA, `ctas` CTAs, n columns.
struct LinTile {
    int ctas, n;
};

// One product for choose_tile(): an m x n result, `depth` 64-deep blocks
// (`split`: which may be split).
struct LinWork {
    int64_t m, n, depth;
    bool split;
};
LinTile choose_tile(LinWork a, LinWork b);

// First words of the workspace, written by the row selection and the combine.
struct LinHeader {
    int64_t n_items;  // rows that count towards the mean
    int32_t n_live;   // rows packed
    float alpha;      // factor of both gradients that is the same for every row
    int32_t dh_splits;  // parts that dhidden's sums came in (grads kernel)
    int32_t done;     // CTAs of the combine that have finished
};

// row_map values of rows that are not packed.
constexpr int32_t kLinRowSkipped = -1;  // masked or ignored: zeros
constexpr int32_t kLinRowBad = -2;      // a target out of range: NaN

struct LinParams {
    const void *hidden, *weight;
    int64_t hidden_stride, weight_stride;  // elements
    int64_t rows, vocab, dim;
    bool bf16;
    const int64_t *targets;  // [rows, k]
    int64_t k;
    bool token_ce;        // k = 1 targets are labels, ignore_index rows are skipped
    bool whole_rows;      // a row with any target out of range is left out whole
    int64_t ignore_index;
    const uint8_t *row_mask;
    float T, c;           // temperature, log2(e) / T

    // forward outputs, by original row (each nullable)
    float *logp_out;      // [rows, k]
    float *state_out;     // [rows, 2] max and sum over the row's columns
    float *loss_rows;     // [rows]
    float *loss_out;      // [1] their sum or mean
    int64_t *n_items_out; // [1]

    // backward
    bool backward;            // the call has gradients
    bool direct;              // a short forward: rows stay where they are, none is packed
    bool fused;               // the statistics were taken by the same call
    const float *grad_out;    // CE: [rows] or [1]; selective: [rows, k]
    int reduction;            // CE: 0 none, 1 sum, 2 mean
    const int64_t *n_items;   // CE mean; null: the header's
    const float *saved_logp, *saved_state;
    void *dhidden, *dweight;  // either may be null
    int64_t dhidden_stride, dweight_stride;
    bool accumulate;          // dweight += instead of =

    // workspace
    LinHeader *head;
    int32_t *row_list, *row_map;  // packed -> original, original -> packed
    int32_t *tgt;                 // [rows_pad, k] packed targets (-1: out of range)
    float *xt;                    // [rows_pad, k] their logits
    float2 *partials;             // [rows_pad, tiles] (max, sum) of each half tile
    float2 *grow;                 // [rows_pad] (M, coef / S)
    float *dzt;                   // [rows_pad, k] dz of the gathered columns
    // Operands of the products are bf16 planes: one for bf16 inputs, three
    // whose sum is the value for fp32 ones.
    int planes;
    int64_t pitch;                // elements from row to row of hpack and wpack
    void *hpack;                  // [planes, rows_pad, pitch] packed live rows
    int64_t hpack_plane;
    bool weight_direct;           // the weight is read in place, else through wpack
    void *wpack;                  // [planes, wpack_rows, pitch] one piece of the weight
    int64_t wpack_rows;
    float *z;                     // [rows_pad, piece] logits kept for the gradient, or null
    void *dz;                     // [planes, rows_pad, piece]
    int64_t dz_plane;
    float *dh;                    // [parts, rows of whole tiles, dh_pitch] sums
    int64_t dh_pitch, dh_room;    // elements from row to row, and in all
    LinTile logits_tile, grads_tile;
    int64_t rows_pad, tiles, piece;
    int64_t stats_warps;          // epilogue warps of the (first) statistics launch

    int32_t *dev_status;
};

// Who makes the gathered columns' logits, fp32 products of two rows each.
// Few: the statistics kernel's epilogue, at most one a warp, while its first
// tile is on its way (48 rows x 4: 34.6 us; after its tiles 36.0).  More: the
// packing before it, a warp each with the memory to itself (2000 x 4096 x 512,
// four targets: 34.6 us; after the tiles 43.5; 7000 x 76032 x 2560, one: 1525
// us either way, before the tiles, behind whose loads they wait, 1569).  The
// warps are those of the CTAs that the launch has, few where tiles are few:
// 300 x 128 x 4096, four targets, six CTAs: in the packing 26 us, after the
// tiles 68; 1000 x 64 x 512, one: 12.6 and 30.6.
inline __host__ __device__ bool lin_dots_in_pack(const LinParams &p)
{
    return !p.direct && (p.fused || !p.backward) && p.rows * p.k > p.stats_warps;
}

cudaError_t lin_select(const LinParams &p, cudaStream_t s);
bool lin_weight_packed(const LinParams &p);  // lin_select packed the weight too
cudaError_t lin_stats(const LinParams &p, cudaStream_t s);
cudaError_t lin_combine(const LinParams &p, cudaStream_t s);
cudaError_t lin_dz(const LinParams &p, cudaStream_t s);
cudaError_t lin_pack_weight(const LinParams &p, int64_t v0, int64_t v1, cudaStream_t s);
cudaError_t lin_grads(const LinParams &p, cudaStream_t s);
cudaError_t lin_finish(const LinParams &p, cudaStream_t s);

}  // namespace gbce
