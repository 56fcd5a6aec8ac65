// Row kernels of the post-training losses over [rows, vocab] logits (sm_103a):
// distillation from a teacher's top logits, and the losses of one token's log
// p per row (the clipped policy loss; the sweeps around the preference loss).
//
// All of them see a row as a few LISTED columns (the teacher's entries; the
// row's token) and the REST.  One sweep takes the online (max m, sum s) of the
// rest with the listed columns left out; the listed logits are gathered on the
// side, so that 1 - p never comes from a difference with 1 (the form of the
// cross-entropy kernels).  The loss and every gradient then follow from (m, s)
// and the listed logits:
//   unlisted j:  dx_j = gs 2^{(x_j - m) c - log2 s}, gs = (g / T) times the
//                rest's whole share of the gradient,
//   listed k:    a value of its own.
//
// A CTA is a ring of bulk copies (one producer thread), NCW consumer warps
// that sweep the copied vectors, and one list warp that is a row ahead: it takes
// the next row, gathers its listed columns while the consumers still sweep the
// row before, and finishes the loss of each swept row.  What bounds it is HBM:
// logits once in, gradients once out; the gradient pass reads its row from L2.
// At 8192 x 152064 bf16, of 6.79 TB/s measured for a copy: distillation with 64
// entries 778 us (0.92), policy loss with 15% of the rows left out 725 us (0.94),
// preference loss of 4096 rows, whose logits are read twice, 490 us (0.93 of the
// bytes it moves).
#pragma once

#include "gbce_kernels.cuh"
#include "gbce_post.h"

namespace gbce {

constexpr float kQuietNan = __builtin_nanf("");

// A value of the problem in two floats (c = log2(e) / T, 1 / T), the first of 14
// bits: products with it do not carry the constant's own rounding.  With c in
// one float log p is off by up to 2e-7 in one direction in every row, and the
// preference loss sums hundreds of them.  Both parts are positive, so that -inf
// times either is -inf.
struct TwoFloat {
    float hi, lo;
};

__device__ __forceinline__ float scaled(float x, TwoFloat k) { return fmaf(x, k.hi, x * k.lo); }

// A sum in two floats: 48 bits without the FP64 units, whose few lanes would set
// the time of a short kernel.
struct Sum2 {
    float hi = 0.0f, lo = 0.0f;

    __device__ __forceinline__ void add(float x)
    {
        const float t = __fadd_rn(hi, x), b = __fsub_rn(t, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(x, b)));
        hi = t;
    }
    __device__ __forceinline__ void add(Sum2 o)
    {
        add(o.hi);
        lo = __fadd_rn(lo, o.lo);
    }
    // a - b, whose rounding error is kept
    __device__ __forceinline__ void add_difference(float a, float b)
    {
        const float d = __fsub_rn(a, b), t = __fsub_rn(d, a);
        add(d);
        lo = __fadd_rn(lo, __fsub_rn(__fsub_rn(a, __fsub_rn(d, t)), __fadd_rn(b, t)));
    }
    // (what a NaN or an infinity leaves in lo says nothing)
    __device__ __forceinline__ double value() const
    {
        return isfinite(hi) ? static_cast<double>(hi) + lo : static_cast<double>(hi);
    }
    __device__ __forceinline__ void warp_merge()
    {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            Sum2 o;
            o.hi = __shfl_down_sync(0xffffffffu, hi, off);
            o.lo = __shfl_down_sync(0xffffffffu, lo, off);
            add(o);
        }
    }
};

// -------------------------------------------------------------- the rest's sum

// The SFU's 2^x is low on the average: by 5.0e-8 of its value for x <= -1, by 2.1e-8
// between -1 and 0, not at all at 0 (measured over 2^20 arguments per unit).  A sum
// over a row would carry that in one direction in every row.  (A mean of one chip's
// units: no bound of the tests rests on it, or on kSumLow.)
constexpr float kEx2Low = 5e-8f;

// 2^x for the factors that whole sums are multiplied by, without it: one more
// step of the last place for three results in four, which is 5.8e-8 on the average.
__device__ __forceinline__ float ex2_level(float x)
{
    const float y = ex2(x);
    return x > -1.0f ? fmaf(y, 2e-8f, y) : fmaf(y, kEx2Low, y);
}

// Online (max, sum) of the unlisted logits in the exp2 domain, as OnlineStats
// but with exponents from both parts of c (one more packed multiply-add per
// pair; the sweep has issue slots to spare).
//
// Far logits, |x| c >= 2^31 (a mask of the type's lowest value, whose x c is not
// even finite): no shift can be taken off them, and none is needed.  Two of them
// that differ do so by 2^7 or more in the exponent, so beside the max only its
// equals count, each 1; the shift stays infinite, which drops what came before.
struct RestStats {
    float m = kNegInf;
    float nmc = __builtin_huge_valf();  // -m c, the shift added to every x c
    float2 sa = make_float2(0.0f, 0.0f);
    float2 sb = make_float2(0.0f, 0.0f);

    // (vmax not far)
    __device__ __forceinline__ void raise_to(float vmax, TwoFloat c)
    {
        if (vmax > m) {
            const float nmc_new = -scaled(vmax, c);
            const float f = ex2(nmc_new - nmc);  // (levelled: 2 to 3% of short rows' time)
            const float2 ff = make_float2(f, f);
            sa = fmul2(sa, ff);
            sb = fmul2(sb, ff);
            m = vmax;
            nmc = nmc_new;
        }
    }
    // A far max (or the one there is) and what was added to it.
    __device__ __forceinline__ void add_far(float2 max_sum)
    {
        if (max_sum.x > m) {
            const float2 zero = make_float2(0.0f, 0.0f);
            sa = fmul2(sa, zero);  // (a NaN stays)
            sb = fmul2(sb, zero);
            m = max_sum.x;
            nmc = m > 0.0f ? kNegInf : __builtin_huge_valf();
        }
        sa.x += max_sum.y;
    }
    // (the large part of x c meets the shift first, where the two cancel: what is
    // rounded is the exponent's own size, and at the max it is residual()'s very steps)
    __device__ __forceinline__ float2 terms(float2 x, TwoFloat c) const
    {
        const float2 hi = make_float2(c.hi, c.hi), lo = make_float2(c.lo, c.lo);
        const float2 z = ffma2(x, lo, ffma2(x, hi, make_float2(nmc, nmc)));
        return make_float2(ex2(z.x), ex2(z.y));
    }
    __device__ __forceinline__ void add(float2 p, float2 q, TwoFloat c)
    {
        sa = fadd2(sa, terms(p, c));
        sb = fadd2(sb, terms(q, c));
    }
    __device__ __forceinline__ void add1(float x, TwoFloat c, float far)
    {
        if (fabsf(x) < far) {
            raise_to(x, c);
            sa.x += ex2(fmaf(x, c.lo, fmaf(x, c.hi, nmc)));
        } else if (x != kNegInf) {
            const float top = x > m ? x : m;
            add_far(make_float2(top, far_term(x, top)));
        }
    }
    // What a logit adds beside a far max `top`: +inf and NaN have no softmax.
    __device__ static __forceinline__ float far_term(float x, float top)
    {
        return x != x || x == __builtin_huge_valf() ? __builtin_nanf("") : (x == top ? 1.0f : 0.0f);
    }
    __device__ __forceinline__ float sum() const
    {
        return __fadd_rn(__fadd_rn(sa.x, sa.y), __fadd_rn(sb.x, sb.y));
    }
    // what every exponent carries of the shift's rounding (OnlineStats::residual)
    __device__ __forceinline__ float residual(TwoFloat c) const
    {
        return isfinite(nmc) ? fmaf(m, c.lo, fmaf(m, c.hi, nmc)) : 0.0f;
    }
};

// Merge the (m, s) of the 32 lanes into one, on every lane, in a fixed order.
__device__ __forceinline__ void warp_merge_rest(float &m, float &s, TwoFloat c, float r = 0.0f)
{
    float M;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(M) : "f"(m));
    float v = 0.0f;
    if (M != kNegInf && m != kNegInf)
        v = __fmul_rn(s, ex2_level(__fsub_rn(scaled(m - M, c), r)));
    m = M;
    s = warp_sum(v);
}

// ... and of two states (the slices of a row, in slice order).
__device__ __forceinline__ void merge_rest(float &m, float &s, float m2, float s2, TwoFloat c)
{
    const float M = fmaxf(m, m2);
    if (M != kNegInf)
        s = __fadd_rn(m == kNegInf ? 0.0f : __fmul_rn(s, ex2_level(scaled(m - M, c))),
                      m2 == kNegInf ? 0.0f : __fmul_rn(s2, ex2_level(scaled(m2 - M, c))));
    m = M;
}

// ------------------------------------------------------------ listed columns

enum RowState : int {
    kRowLive = 0,
    kRowSkip = 1,     // left out, or a teacher without mass: loss 0, gradient 0
    kRowInvalid = 2,  // NaN outputs (a bad index or label, a NaN teacher logit)
    kRowEnd = 3,      // no more rows
};

// One row on its way through a CTA: what the list warp found out about it.
struct RowSlot {
    int64_t r;
    int early;     // RowState as far as the label, the mask and the columns tell
    int state;     // ... and the teacher
    int streamed;  // the producer copies the row
    float m, s;    // the rest's state: from the consumers (or, backward, for them)
    float gt;      // upstream gradient / T
    // distill: listed logits' max, and sum of 2^{(x - ml) c} without one holder of the
    // max; teacher's log p of the unlisted columns (-inf: none)
    float ml, sl, lp_rest;
    // token: column, logit; advantage, old and reference log p
    int y;
    float xy, adv, old_lp, ref_lp;
    float dy;  // token: the gradient at its column
};

// The listed columns of a row, in shared memory.  Column col of a row is owned
// by one consumer thread (the one whose sweep reads it); the entries of an owner
// form a chain head[owner] -> next -> ... of which a thread walks only its own,
// so that leaving them out of the sweep needs no barrier between threads.
struct ListRef {
    int32_t *head;  // [NC]
    int32_t *col;   // [k] column; -1: no entry; -2 - column: a repeat of an earlier one
    int32_t *next;  // [k]
    float *x;       // [k] student logit
    float *lp;      // [k] teacher's log p
    float *val;     // [k] gradient at the column
};

__host__ __device__ __forceinline__ int list_words(int nc, int k) { return nc + 5 * k; }

__device__ __forceinline__ ListRef list_at(int32_t *words, int nc, int k)
{
    ListRef L;
    L.head = words;
    L.col = words + nc;
    L.next = L.col + k;
    L.x = reinterpret_cast<float *>(L.next + k);
    L.lp = L.x + k;
    L.val = L.lp + k;
    return L;
}

// Which part of a row a CTA sweeps.
struct Slice {
    RowGeom g;
    int64_t v0, v1;    // body vectors
    bool first, last;  // the slice holds the row's scalar head / tail
};

template <int VEC, int NC>
__device__ __forceinline__ int column_owner(const Slice &sl, int32_t col)
{
    if (col < sl.g.head)
        return col;
    if (col >= sl.g.tail0)
        return static_cast<int>(col - sl.g.tail0);
    // (a column of another slice has an owner too: its entry is found there by
    // the search for repeats, and its vector lies outside [v0, v1))
    const int32_t v = (col - static_cast<int32_t>(sl.g.head)) / VEC - static_cast<int32_t>(sl.v0);
    const int32_t o = v % NC;
    return o < 0 ? o + NC : o;
}

// (this lane's value, its entry) -> the warp's largest value and the lowest
// entry that has it (INT32_MAX when the value is -inf everywhere)
__device__ __forceinline__ void warp_argmax(float &v, int32_t &k)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float v2 = __shfl_xor_sync(0xffffffffu, v, off);
        const int32_t k2 = __shfl_xor_sync(0xffffffffu, k, off);
        if (v2 > v || (v2 == v && k2 < k)) {
            v = v2;
            k = k2;
        }
    }
}

constexpr int kBatch = 4;  // entries that a lane loads at a time

// The columns of row r's entries and their chains (one warp): what the sweep
// needs.  An index listed twice is one column: the first entry keeps it and has
// its bit set in `repeated` (this lane's entry lane + 32 i: bit i).  Returns
// whether an index is out of range.
template <typename T, int NC>
__device__ bool list_columns(const PostParams &p, int64_t r, const Slice &sl, const ListRef &L,
                             int lane, uint32_t &repeated)
{
    constexpr int VEC = Elem<T>::kVec;
    const int K = static_cast<int>(p.k);
    const int64_t *index = p.index + r * K;
    bool bad = false;
    for (int i = lane; i < NC; i += 32)
        L.head[i] = -1;
    // (kBatch loads of a lane in flight together: one memory latency, not K / 32)
    for (int k0 = lane; k0 < K; k0 += 32 * kBatch) {
        int64_t t[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
            t[b] = k0 + 32 * b < K ? __ldg(index + k0 + 32 * b) : -1;
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const bool here = t[b] >= 0 && t[b] < p.vocab;
            bad |= !here && t[b] != -1;
            if (k0 + 32 * b < K)
                L.col[k0 + 32 * b] = here ? static_cast<int32_t>(t[b]) : -1;
        }
    }
    bad = __any_sync(0xffffffffu, bad);
    __syncwarp();
#pragma unroll 4
    for (int k = lane; k < K; k += 32)
        if (L.col[k] >= 0)
            L.next[k] = atomicExch(&L.head[column_owner<VEC, NC>(sl, L.col[k])], k);
    __syncwarp();
    // Repeats: equal columns share an owner, so its chain shows them all, each
    // pair to the one of the two that was put in later.  There are none as a rule.
    bool same = false;
#pragma unroll 4
    for (int k = lane; k < K; k += 32) {
        const int32_t col = L.col[k];
        if (col >= 0)
            for (int j = L.next[k]; j >= 0; j = L.next[j])
                same |= L.col[j] == col;
    }
    repeated = 0;
    if (!__any_sync(0xffffffffu, same))
        return bad;
    uint32_t repeat = 0;
    for (int k = lane, i = 0; k < K; k += 32, ++i) {
        const int32_t col = L.col[k];
        if (col < 0)
            continue;
        for (int j = L.head[column_owner<VEC, NC>(sl, col)]; j >= 0; j = L.next[j])
            if (j != k && L.col[j] == col)
                (j < k ? repeat : repeated) |= 1u << i;
    }
    repeated &= ~repeat;
    __syncwarp();
    for (int k = lane, i = 0; k < K; k += 32, ++i)
        if (repeat >> i & 1u)
            L.col[k] = -2 - L.col[k];
    return bad;
}

// A teacher's logit / T.  One that is finite stays so (a mask of the lowest value,
// T < 1): entries that are all as low still share their mass.
__device__ __forceinline__ float teacher_logit(float raw, TwoFloat inv_t)
{
    return raw == kNegInf ? kNegInf : fmaxf(scaled(raw, inv_t), -3.402823466e38f);
}

// ... relative to the list's largest, and the rest's then: a list that names a column
// twice adds log 2 to some of its logits, which one of 1e38 would swallow.
__device__ __forceinline__ float teacher_logit(float raw, float top, TwoFloat inv_t)
{
    return raw == kNegInf ? kNegInf : scaled(raw - top, inv_t);
}
__device__ __forceinline__ float rest_logit(float rest, float top, TwoFloat inv_t)
{
    return rest == kNegInf || top == kNegInf
               ? rest
               : fminf(rest - teacher_logit(top, inv_t), 3.402823466e38f);
}

// Bring a row's entries into L2.
__device__ __forceinline__ void prefetch_entries(const PostParams &p, int64_t r, int lane)
{
    const auto line = [&](const void *base, int64_t bytes, int i) {
        const int64_t at = 128 * static_cast<int64_t>(i) < bytes ? 128 * i : bytes - 1;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char *>(base) + at));
    };
    // (256 entries: 17 lines of columns at most, 9 of logits)
    if (lane < 18)
        line(p.index + r * p.k, p.k * 8, lane);
    else if (lane < 28)
        line(p.teacher + r * p.k, p.k * 4, lane - 18);
    else if (lane == 28 && p.teacher_rest != nullptr)
        line(p.teacher_rest + r, 4, 0);
}

// The teacher's distribution, the softmax over its logits / T and teacher_rest,
// and the student's logits at its columns (one warp, after list_columns).
// A NaN or +inf among the teacher's logits makes the row invalid.
template <typename T>
__device__ void list_teacher(const PostParams &p, int64_t r, const T *row, const ListRef &L,
                             RowSlot &slot, int lane, uint32_t repeated)
{
    const int K = static_cast<int>(p.k);
    const TwoFloat c = {p.c_hi, p.c_lo}, inv_t = {p.it_hi, p.it_lo};
    const float inf = __builtin_huge_valf();
    const float *teacher = p.teacher + r * K;
    float rest = p.teacher_rest != nullptr ? p.teacher_rest[r] : kNegInf;
    bool nan_t = !(rest < inf);
    for (int k0 = lane; k0 < K; k0 += 32 * kBatch) {
        float raw[kBatch], x[kBatch];
        bool in[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int k = k0 + 32 * b;
            const int32_t col = k < K ? L.col[k] : -1;
            in[b] = col >= 0;
            raw[b] = in[b] ? __ldg(teacher + k) : kNegInf;
            x[b] = in[b] ? Elem<T>::load(row + col) : kNegInf;
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int k = k0 + 32 * b;
            nan_t |= in[b] && !(raw[b] < inf);
            if (k < K) {
                L.x[k] = x[b];
                L.lp[k] = teacher_logit(raw[b], inv_t);
            }
        }
    }
    if (__any_sync(0xffffffffu, repeated != 0)) {
        // the first of several takes their sum, in entry order
        float top = kNegInf;
        for (int k = 0; k < K; ++k)
            if (L.col[k] != -1) {
                nan_t |= !(teacher[k] < inf);
                top = fmaxf(top, teacher[k]);
            }
        rest = rest_logit(rest, top, inv_t);
        for (int k = lane, i = 0; k < K; k += 32, ++i) {
            const int32_t col = L.col[k];
            if (col < 0)
                continue;
            L.lp[k] = teacher_logit(teacher[k], top, inv_t);
            if (!(repeated >> i & 1u))
                continue;
            const auto tau = [&](int j) {
                return L.col[j] == col || L.col[j] == -2 - col ? teacher_logit(teacher[j], top, inv_t)
                                                               : kNegInf;
            };
            float m = kNegInf, s = 0.0f;
            for (int j = k; j < K; ++j)
                m = fmaxf(m, tau(j));
            for (int j = k; j < K; ++j)
                if (tau(j) != kNegInf)
                    s += expf(tau(j) - m);
            L.lp[k] = s > 0.0f ? m + logf(s) : kNegInf;
        }
    }
    nan_t = __any_sync(0xffffffffu, nan_t);
    // maxima: the teacher's over the entries and the rest, the student's
    float mt = kNegInf, ml = kNegInf;
    int32_t at = INT32_MAX, al = INT32_MAX;
    bool nan_x = false;
    for (int k = lane; k < K; k += 32) {
        if (L.col[k] < 0)
            continue;
        const float tau = L.lp[k], x = L.x[k];
        if (tau > mt) {
            mt = tau;
            at = k;
        }
        nan_x |= x != x || x == inf;
        if (x > ml) {
            ml = x;
            al = k;
        }
    }
    warp_argmax(mt, at);
    warp_argmax(ml, al);
    nan_x = __any_sync(0xffffffffu, nan_x);
    if (rest > mt) {
        mt = rest;
        at = -1;
    }
    // the sums without one holder of the maximum, whose own term is 1
    float st = (lane == 0 && at != -1 && rest != kNegInf) ? expf(rest - mt) : 0.0f, sx = 0.0f;
    for (int k = lane; k < K; k += 32) {
        if (L.col[k] < 0)
            continue;
        if (k != at && L.lp[k] != kNegInf)
            st += expf(L.lp[k] - mt);
        if (k != al && L.x[k] != kNegInf)
            sx += ex2(scaled(L.x[k] - ml, c));
    }
    st = warp_sum(st);
    sx = warp_sum(sx);
    const float lt = log1pf(st);
    for (int k = lane; k < K; k += 32)
        L.lp[k] = (L.lp[k] - mt) - lt;
    if (lane == 0) {
        // a row with a NaN (or +inf) listed logit has no softmax
        slot.ml = nan_x ? 0.0f : ml;
        slot.sl = nan_x ? kQuietNan : sx;
        slot.lp_rest = rest == kNegInf ? kNegInf : (rest - mt) - lt;
        slot.state = nan_t ? kRowInvalid : (mt == kNegInf ? kRowSkip : kRowLive);
    }
}

// ------------------------------------------------------- distillation of a row

// The student's softmax from the rest's state (m, s) and the listed logits'
// (ml, sl): log q_k = (x_k - M) / T - log_s, and log q of the rest.
struct StudentRow {
    float M, log_s, log_rest;
};

__device__ __forceinline__ StudentRow student_row(float m, float s, float ml, float sl, TwoFloat c,
                                                  TwoFloat inv_t)
{
    StudentRow q;
    q.M = fmaxf(m, ml);
    const float rest = m == kNegInf ? s : s * ex2(scaled(m - q.M, c));
    const float listed = ml == kNegInf ? 0.0f : (1.0f + sl) * ex2(scaled(ml - q.M, c));
    // log of the whole sum: past its own largest term where that is listed
    q.log_s = ml >= m ? log1pf(sl + rest) : logf(rest + listed);
    // log of the rest's share, by whichever of the two does not cancel
    q.log_rest = rest >= listed
                     ? -log1pf(listed / rest)
                     : (s > 0.0f ? (logf(s) + scaled(m - q.M, inv_t)) - q.log_s : kNegInf);
    if (q.M == kNegInf || listed != listed || rest != rest)
        q.log_s = q.log_rest = kQuietNan;
    return q;
}

// (e^u - 1 - u) / u^2 for |u| < 1/2, by its series: the next term is below
// 2^-28 of the sum.
__device__ __forceinline__ float phi_series(float u)
{
    float h = 1.0f / 362880.0f;
    h = fmaf(h, u, 1.0f / 40320.0f);
    h = fmaf(h, u, 1.0f / 5040.0f);
    h = fmaf(h, u, 1.0f / 720.0f);
    h = fmaf(h, u, 1.0f / 120.0f);
    h = fmaf(h, u, 1.0f / 24.0f);
    h = fmaf(h, u, 1.0f / 6.0f);
    return fmaf(h, u, 0.5f);
}

// One entry of the two distributions (p teacher, q student), u = log q - log p:
//  kl   p phi(u), phi(u) = e^u - 1 - u >= 0: one term of KL = sum p (log p -
//       log q) written as a sum of non-negative terms (both distributions sum to
//       1, so the extra q - p sum to 0);
//  gap  q - p.
// Near u = 0 both come from phi's series: a near-converged student keeps its
// loss and gradient, where the plain terms cancel to fp32's rounding (beyond, the
// differences cancel a factor of 17 and 4 at most).
struct EntryTerms {
    float kl, gap;
};

__device__ __forceinline__ EntryTerms entry_terms(float lp, float lq)
{
    const float p = expf(lp), q = expf(lq), u = lq - lp;
    const float near = u * phi_series(u);
    const bool close = fabsf(u) < 0.5f;
    EntryTerms t;
    t.gap = close ? p * fmaf(u, near, u) : q - p;
    t.kl = close ? p * (u * near) : (q - p) - p * u;
    if (!(p > 0.0f) && p == p) {  // (0 log 0 = 0)
        t.kl = q;
        t.gap = q;
    }
    return t;
}

// q_rest - p_rest.  Every consumer thread waits for it between its two sweeps, so
// the usual teacher, one without a rest, takes q_rest as the plain quotient.
__device__ __forceinline__ float rest_gap(float m, float s, float ml, float sl, float lp_rest,
                                          TwoFloat c, TwoFloat inv_t)
{
    if (lp_rest != kNegInf)
        return entry_terms(lp_rest, student_row(m, s, ml, sl, c, inv_t).log_rest).gap;
    const float M = fmaxf(m, ml);
    const float rest = m == kNegInf ? s : s * ex2(scaled(m - M, c));
    const float listed = ml == kNegInf ? 0.0f : (1.0f + sl) * ex2(scaled(ml - M, c));
    return __fdividef(rest, rest + listed);
}

__device__ __forceinline__ float student_logp(const StudentRow &q, float x, TwoFloat inv_t)
{
    return scaled(x - q.M, inv_t) - q.log_s;
}

// ----------------------------------------------------- one token's log p

// What is left in a sum of what its terms' 2^x lacks: the factors, levelled two or
// three times, overshoot by 8e-9 each.  With it log p of 1000 to 4000 rows of 100 to
// 152064 logits, T 0.7 to 2, lies -4e-8 to 5e-8 of 1 - p from fp64's on the average, half
// of its scatter (0.8e-7 to 1.8e-7) or less.
constexpr float kSumLow = 3.5e-8f;

// log p of one column from the rest's (m, s): -log(1 + e^a), a = log s + (m - xy) / T,
// with a in two floats throughout: log s from its exponent and mantissa, the
// quotient with what its products round off.  A preference loss sums hundreds of
// these, and in one float a alone is off by 2.5e-7 (rms) before log p is rounded.
struct TokenTerms {
    float lp, other;  // log p, 1 - p
};

__device__ __forceinline__ TokenTerms token_terms(float m, float s, float xy, TwoFloat inv_t)
{
    // nothing beside the label: certain, if the label itself is anything; a label of
    // +inf, or a row that is -inf throughout, has no softmax
    if (!(s > 0.0f) || xy == __builtin_huge_valf()) {
        const float v = s == 0.0f && isfinite(xy) ? 0.0f : kQuietNan;
        return {v, v};
    }
    // s = 2^k f, f in [1, 2): log s = k log 2 + log f, k log 2 exact in its first part
    // (14 bits of log 2)
    const uint32_t bits = __float_as_uint(s);
    const bool split = bits >= 0x00800000u && bits < 0x7f800000u;  // (normal)
    const int k = split ? static_cast<int>(bits >> 23) - 127 : 0;
    const float f = split ? __uint_as_float((bits & 0x007fffffu) | 0x3f800000u) : s;
    const float k_hi = k * 0x1.62e4p-1f, rest = fmaf(k, 0x1.7f7d1cp-20f, logf(f));
    // d = (m - xy) / T
    const float gap = __fsub_rn(m, xy), gap_lo = __fsub_rn(__fsub_rn(m, gap), xy);
    const float d = scaled(gap, inv_t);
    const float d_lo = fmaf(gap, inv_t.hi, -d) + fmaf(gap, inv_t.lo, gap_lo * inv_t.hi);
    // a = hi + lo
    const float t = __fadd_rn(k_hi, d), b = __fsub_rn(t, k_hi);
    if (!isfinite(t) || !split) {
        const float lp = -softplus(t + rest);
        return {lp, -expm1f(lp)};
    }
    const float small =
        __fadd_rn(__fsub_rn(k_hi, __fsub_rn(t, b)), __fsub_rn(d, b)) +
        (d_lo + (kSumLow - __fdividef(kSumLow, s)) + rest);  // (the largest term is 1 exactly)
    const float hi = __fadd_rn(t, small), lo = __fsub_rn(small, __fsub_rn(hi, t));
    const float e = expf(-fabsf(hi)), sig = __fdividef(e, 1.0f + e);  // sigma(-|a|)
    if (hi > 0.0f)
        return {-(hi + (log1pf(e) + (lo - lo * sig))), 1.0f - sig};
    return {-(log1pf(e) + lo * sig), sig};
}

// The clipped policy loss of one row from its log p, and its derivative:
//   rho = e^{lp - old},  loss = -min(rho A, clip(rho) A) + beta (e^d - 1 - d),
//   d = ref - lp;  d loss / d lp = -rho A [not clipped] - beta (e^d - 1).
// At a clip's border the unclipped side is taken.
__device__ __forceinline__ void policy_row(const PolicyTerms &t, float A, float old_lp,
                                           float ref_lp, float lp, float &loss, float &dlp)
{
    loss = dlp = lp != lp ? kQuietNan : 0.0f;
    if (A != 0.0f && lp == lp) {  // (no advantage: no surrogate, however large the ratio)
        const float rho = t.old_logp != nullptr ? expf(lp - old_lp) : 1.0f;
        const float edge = A > 0.0f ? 1.0f + t.clip_high : 1.0f - t.clip_low;
        const bool held = A > 0.0f ? rho > edge : rho < edge;
        loss = -A * (held ? edge : rho);
        dlp = held ? 0.0f : -A * rho;
        if (rho != rho || A != A)
            loss = dlp = kQuietNan;
    }
    if (t.ref_logp != nullptr && t.kl_beta != 0.0f) {
        const float d = ref_lp - lp, e = expm1f(d);
        const float k3 = fabsf(d) < 0.5f ? d * d * phi_series(d) : e - d;
        loss = fmaf(t.kl_beta, k3, loss);
        dlp = fmaf(-t.kl_beta, e, dlp);
    }
}

// ------------------------------------------------------------- the gradient

// Constants of the sweep over the unlisted columns: gs 2^{(x - m) c - log2 s}.
// Every exponent is <= 0 and relative to the rest's own max, so no element
// carries the rounding of a large offset.  The bf16 sweep adds the offset to x c in
// one step: what kbx rounds off goes into gs, and c is taken smaller where m c would
// pass 2^30 (two bf16 logits that differ are 2^22 apart there, whatever c is).
template <typename T>
__device__ __forceinline__ GradConsts rest_consts(float m, float s, float c, float gs)
{
    const bool none = !(s > 0.0f) || !isfinite(m);  // nothing unlisted has mass
    GradConsts k;
    k.off = 0.0f;
    k.nxy = none ? 0.0f : -m;
    k.c = sizeof(T) == 2 && !none ? fminf(c, 0x1p30f / fabsf(m)) : c;
    k.kb = none ? 0.0f : -log2f(s);
    k.kbx = none ? 0.0f : fmaf(-m, k.c, k.kb);
    k.gs = none && s == s && gs == gs && m != __builtin_huge_valf() ? 0.0f : gs;
    if (sizeof(T) == 2 && !none) {
        const float kept = fmaf(m, k.c, k.kbx);  // kb as kbx has it
        k.gs *= ex2(k.kb - kept);
        k.kb = kept;
    }
    k.dy = 0.0f;
    k.c0 = 0.0f;
    k.ea = k.eb = 0.0f;
    return k;
}

__device__ __forceinline__ float post_upstream(const PostParams &p, int64_t r, int64_t n)
{
    if (p.reduction == 0)
        return p.grad_out[r];
    if (p.reduction == 1)
        return p.grad_out[0];
    return n > 0 ? p.grad_out[0] / static_cast<float>(n) : 0.0f;
}

// ------------------------------------------------------------ the row kernel

// The row that is swept, and the one after it.
constexpr int kRowSlots = 2;

// Consumer warps and ring of the three CTA shapes (see post_shape).
template <int SHAPE> struct PostShape;
template <> struct PostShape<kShapeLong> {
    static constexpr int kWarps = 24, kChunk = 49152, kStages = 4, kCtasPerSm = 1;
};
template <> struct PostShape<kShapeMid> {
    static constexpr int kWarps = 8, kChunk = 16384, kStages = 4, kCtasPerSm = 3;
};
template <> struct PostShape<kShapeShort> {
    static constexpr int kWarps = 4, kChunk = 16384, kStages = 2, kCtasPerSm = 5;
};

template <int SHAPE> constexpr int post_threads() { return (PostShape<SHAPE>::kWarps + 2) * 32; }

template <int SHAPE> constexpr int post_smem(int op, int64_t k)
{
    using S = PostShape<SHAPE>;
    return S::kStages * (S::kChunk + kRingAlign) + kRingAlign +
           (op == kOpDistill
                ? kRowSlots * 4 * list_words(S::kWarps * 32, static_cast<int>(k))
                : 0);
}

// Fold one vector into a thread's rest state.
__device__ __forceinline__ void rest_add(RestStats &st, const uint4 &a, TwoFloat c,
                                         const __nv_bfloat16 *)
{
    st.add(bf16x2_to_float2(a.x), bf16x2_to_float2(a.y), c);
    st.add(bf16x2_to_float2(a.z), bf16x2_to_float2(a.w), c);
}

__device__ __forceinline__ void rest_add(RestStats &st, const uint4 &a, TwoFloat c, const float *)
{
    st.add(make_float2(__uint_as_float(a.x), __uint_as_float(a.y)),
           make_float2(__uint_as_float(a.z), __uint_as_float(a.w)), c);
}

__device__ __forceinline__ uint4 all_neg_inf(float)
{
    return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
}
__device__ __forceinline__ uint4 all_neg_inf(__nv_bfloat16)
{
    return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
}

// Two vectors whose largest logit is far, NaN or -inf, beside a max m: the new max,
// and what they add to it.  Out of line, for few are and the sweeps' loops stay short.
template <typename T> static __device__ __noinline__ float2 far_pair(uint4 a, uint4 b, float m, float far)
{
    constexpr int VEC = Elem<T>::kVec;
    const float top = FastVec<T>::vmax(a, b);
    if (top == kNegInf) {
        // nothing, unless there are NaN, which a max passes over
        const uint32_t none = all_neg_inf(T()).x;
        const uint32_t other = (a.x ^ none) | (a.y ^ none) | (a.z ^ none) | (a.w ^ none) |
                               (b.x ^ none) | (b.y ^ none) | (b.z ^ none) | (b.w ^ none);
        return make_float2(m, other == 0 ? 0.0f : kQuietNan);
    }
    // (a top that is not far lies beside another thread's far one, which drops it)
    const float M = top > m && fabsf(top) >= far ? top : m;
    float f[VEC], g[VEC], s = 0.0f;
    Elem<T>::unpack(a, f);
    Elem<T>::unpack(b, g);
#pragma unroll
    for (int e = 0; e < VEC; ++e)
        s += RestStats::far_term(f[e], M) + RestStats::far_term(g[e], M);
    return make_float2(M, s);
}

// One vector, and two with `top` the largest of them, or of the warp's.
template <typename T>
__device__ __forceinline__ void rest_take(RestStats &st, const uint4 &a, TwoFloat c, float far)
{
    const float top = FastVec<T>::vmax(a);
    if (fabsf(top) < far) {
        st.raise_to(top, c);
        rest_add(st, a, c, static_cast<const T *>(nullptr));
    } else {
        st.add_far(far_pair<T>(a, all_neg_inf(T()), st.m, far));
    }
}

template <typename T>
__device__ __forceinline__ void rest_take(RestStats &st, const uint4 &a, const uint4 &b, float top,
                                          TwoFloat c, float far)
{
    if (fabsf(top) < far) {
        st.raise_to(top, c);
        rest_add(st, a, c, static_cast<const T *>(nullptr));
        rest_add(st, b, c, static_cast<const T *>(nullptr));
    } else {
        st.add_far(far_pair<T>(a, b, st.m, far));
    }
}

// Orders the consumers' writes to a stage (which the release of the stage has
// made this thread see) before the bulk copy that refills it.
__device__ __forceinline__ void fence_before_refill()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ float neg_inf_as(float) { return kNegInf; }
__device__ __forceinline__ __nv_bfloat16 neg_inf_as(__nv_bfloat16)
{
    return __ushort_as_bfloat16(0xff80);
}

// The VEC elements that begin `sh` elements into the pair (a, b).
template <typename T>
__device__ __forceinline__ uint4 shifted(uint4 a, uint4 b, int sh)
{
    const int words = sizeof(T) == 2 ? sh >> 1 : sh;
    if (words & 1) {
        a = make_uint4(a.y, a.z, a.w, b.x);
        b = make_uint4(b.y, b.z, b.w, b.w);
    }
    if (words & 2) {
        a = make_uint4(a.z, a.w, b.x, b.y);
        b.x = b.z;
    }
    if (sizeof(T) == 2 && (sh & 1))
        a = make_uint4(__funnelshift_r(a.x, a.y, 16), __funnelshift_r(a.y, a.z, 16),
                       __funnelshift_r(a.z, a.w, 16), __funnelshift_r(a.w, b.x, 16));
    return a;
}

// How a gradient row is stored: 16-byte vectors from element `begin` on, whose
// elements begin `sh` elements into a logits vector.  sh = 0: the two rows share
// their phase, and vector v of the one is vector v of the other.  Otherwise
// vector v is made of the logits vectors v and v + 1, and the elements before
// the first and behind the last such pair are stored one by one.
struct StoreGeom {
    int sh;
    int64_t begin, vecs, end;  // scalars [0, begin) and [end, V)
};

template <typename T>
__device__ __forceinline__ StoreGeom store_geom(const T *drow, const RowGeom &g, int64_t V)
{
    constexpr int VEC = Elem<T>::kVec;
    const int dhead = static_cast<int>(
        ((16u - static_cast<uint32_t>(reinterpret_cast<uintptr_t>(drow) & 15u)) & 15u) / sizeof(T));
    StoreGeom d;
    d.sh = static_cast<int>(dhead - g.head) & (VEC - 1);
    if (d.sh == 0) {
        d.begin = g.head;
        d.vecs = g.nvec;
    } else {
        d.vecs = g.nvec > 1 ? g.nvec - 1 : 0;
        d.begin = d.vecs > 0 ? g.head + d.sh : V;
    }
    d.end = d.begin + d.vecs * VEC;
    return d;
}

// The columns of a gradient row that a slice's CTA stores.
struct StoredRange {
    int32_t vecs;    // vectors
    int64_t lo, hi;  // columns
};

template <int VEC>
__device__ __forceinline__ StoredRange stored_range(const Slice &sl, const StoreGeom &d, int64_t V)
{
    const int64_t here = d.vecs - sl.v0, most = sl.v1 - sl.v0;
    const int64_t first = sl.g.head + d.sh + sl.v0 * VEC;
    StoredRange t;
    t.vecs = static_cast<int32_t>(here < most ? (here > 0 ? here : 0) : most);
    t.lo = sl.first ? 0 : first;
    t.hi = sl.last ? V : first + static_cast<int64_t>(t.vecs) * VEC;
    return t;
}

template <typename T, int OP, int PASS, int SHAPE>
__global__ void __launch_bounds__(post_threads<SHAPE>(), PostShape<SHAPE>::kCtasPerSm)
    post_kernel(const PostParams p)
{
    using E = Elem<T>;
    using Shape = PostShape<SHAPE>;
    constexpr int VEC = E::kVec;
    constexpr int NCW = Shape::kWarps, NC = NCW * 32;
    constexpr int S = Shape::kStages, CHUNK = Shape::kChunk, CV = CHUNK / 16;
    constexpr int PITCH = CHUNK + kRingAlign;  // of the stages: a chunk and one vector more
    constexpr int PER_THREAD = CV / NC, Q = kRowSlots;
    static_assert(CV % NC == 0 && PER_THREAD % 2 == 0, "a chunk splits into pairs of vectors");
    constexpr bool kStats = PASS != kPassBwd, kGrad = PASS != kPassFwd;
    constexpr int kPasses = (kStats ? 1 : 0) + (kGrad ? 1 : 0);
    constexpr bool kList = OP == kOpDistill;

    extern __shared__ __align__(128) uint8_t dyn_smem[];
    uint8_t *ring = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(dyn_smem) + (kRingAlign - 1)) & ~uintptr_t(kRingAlign - 1));
    int32_t *lists = reinterpret_cast<int32_t *>(ring + S * PITCH);
    __shared__ uint64_t full_bar[S], empty_bar[S];
    // rows: known (to the producer), columns known and all else known (to the
    // consumers), statistics done (to the list warp), slot free again
    __shared__ uint64_t row_bar[Q], cols_bar[Q], list_bar[Q], stat_bar[Q], free_bar[Q];
    __shared__ RowSlot slots[Q];
    // per-warp partials, double-buffered by swept row: a warp that has merged one
    // row can write the next one's while a slower warp still reads (rows that are
    // not swept have no barrier, so they do not count)
    __shared__ float red_m[2][NCW], red_s[2][NCW];
    __shared__ uint64_t xbar;  // cluster of CTAs per row: every slice's partial
    __shared__ __align__(16) float4 xchg[kMaxClusterCtas];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t V = p.vocab;
    const TwoFloat c = {p.c_hi, p.c_lo}, inv_t = {p.it_hi, p.it_lo};
    const int C = p.splits;
    const int64_t cluster = C > 1 ? blockIdx.x / C : blockIdx.x;
    const int split = C > 1 ? static_cast<int>(blockIdx.x - cluster * C) : 0;
    const int64_t clusters = gridDim.x / C;

    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full_bar[i], 1);
            mbar_init(&empty_bar[i], NCW);
        }
        for (int i = 0; i < Q; ++i) {
            mbar_init(&row_bar[i], 1);
            mbar_init(&cols_bar[i], 1);
            mbar_init(&list_bar[i], 1);
            mbar_init(&stat_bar[i], 1);
            mbar_init(&free_bar[i], NCW + 1);
        }
        mbar_init(&xbar, 1);
        fence_barrier_init();
    }
    __syncthreads();
    if (C > 1)
        cluster_arrive_relaxed();
    // With a ticket, the kernel before this one is the library's own count (or
    // clearing), which starts only once everything before it is complete: the
    // first row does not wait for it, only what it wrote does (list warp).
    // Otherwise it is the caller's, and may still be writing what is read here.
    if (p.ticket == nullptr)
        grid_dependency_wait();

    const auto slice_of = [&](const T *row) {
        Slice sl;
        sl.g = row_geom<T>(row, V);
        sl.v0 = C == 1 ? 0 : sl.g.nvec * split / C;
        sl.v1 = C == 1 ? sl.g.nvec : sl.g.nvec * (split + 1) / C;
        sl.first = split == 0;
        sl.last = split == C - 1;
        return sl;
    };

    // ------------------------------------------------------------ list warp
    if (warp == NCW + 1) {
        bool ok = true;
        const auto list_of = [&](int q) {
            return list_at(lists + q * list_words(NC, static_cast<int>(p.k)), NC,
                           static_cast<int>(p.k));
        };
        // what follows from row i's statistics: its loss (by the first slice's
        // CTA), and the gradients at its listed columns
        const auto finish = [&](uint32_t i) {
            const int q = i % Q;
            RowSlot &w = slots[q];
            if (w.state != kRowLive) {
                if (kStats && lane == 0 && split == 0) {
                    const float fill = w.state == kRowSkip ? 0.0f : kQuietNan;
                    if (p.loss_rows != nullptr)
                        p.loss_rows[w.r] = fill;
                    if (p.logp_out != nullptr)
                        p.logp_out[w.r] = fill;
                    if (p.rest_state_out != nullptr) {
                        p.rest_state_out[2 * w.r] = kNegInf;
                        p.rest_state_out[2 * w.r + 1] = 0.0f;
                    }
                }
                return;
            }
            if (kStats && !mbar_wait(&stat_bar[q], (i / Q) & 1)) {
                ok = false;
                return;
            }
            const float m = w.m, s = w.s;
            if (kStats && p.rest_state_out != nullptr && lane == 0 && split == 0) {
                p.rest_state_out[2 * w.r] = m;
                p.rest_state_out[2 * w.r + 1] = s;
            }
            if (kList) {
                const ListRef L = list_of(q);
                const StudentRow st = student_row(m, s, w.ml, w.sl, c, inv_t);
                float kl = lane == 0 ? entry_terms(w.lp_rest, st.log_rest).kl : 0.0f;
#pragma unroll 2
                for (int k = lane; k < p.k; k += 32) {
                    if (L.col[k] < 0)
                        continue;
                    const EntryTerms t =
                        entry_terms(L.lp[k], student_logp(st, L.x[k], inv_t));
                    kl += t.kl;
                    if (kGrad)
                        L.val[k] = w.gt * t.gap;
                }
                kl = warp_sum(kl);
                if (kStats && lane == 0 && split == 0)
                    p.loss_rows[w.r] = kl;
            } else if (lane == 0) {
                const TokenTerms y = token_terms(m, s, w.xy, inv_t);
                float slope = w.gt;
                if (kStats && p.logp_out != nullptr && split == 0)
                    p.logp_out[w.r] = y.lp;
                if (OP == kOpPolicy) {
                    float loss, dlp;
                    policy_row(p.policy, w.adv, w.old_lp, w.ref_lp, y.lp, loss, dlp);
                    if (split == 0)
                        p.loss_rows[w.r] = loss;
                    slope *= dlp;
                }
                if (kGrad)
                    w.dy = slope * y.other;
            }
        };
        // row i's listed columns, over what the sweep stored there (every thread
        // of this CTA has stored its part: the slot is free)
        const auto patch = [&](uint32_t i) {
            const int q = i % Q;
            const RowSlot &w = slots[q];
            if (!kGrad || w.state != kRowLive)
                return;
            const T *row = static_cast<const T *>(p.logits) + w.r * p.row_stride;
            T *drow = static_cast<T *>(p.dlogits) + w.r * p.d_stride;
            const Slice sl = slice_of(row);
            const StoreGeom dg = store_geom<T>(drow, sl.g, V);
            const StoredRange range = stored_range<VEC>(sl, dg, V);
            if (kList) {
                const ListRef L = list_of(q);
                for (int k = lane; k < p.k; k += 32)
                    if (L.col[k] >= range.lo && L.col[k] < range.hi)
                        E::store(drow + L.col[k], L.val[k]);
            } else if (lane == 0 && w.y >= range.lo && w.y < range.hi) {
                E::store(drow + w.y, w.dy);
            }
        };
        // row i is done when its slot is free: then its patches, and the slot is
        // this warp's again
        const auto retire = [&](uint32_t i) {
            finish(i);
            __syncwarp();
            if (ok && !mbar_wait(&free_bar[i % Q], (i / Q) & 1))
                ok = false;
            if (ok)
                patch(i);
            __syncwarp();
            return ok;
        };
        const int64_t lo = p.row_range != nullptr ? p.row_range[0] : 0;
        const int64_t hi = p.row_range != nullptr ? p.row_range[p.row_range_end] : p.rows;
        const auto row_at = [&](int64_t t) { return p.reverse ? p.rows - 1 - t : t; };
        const auto key_of = [&](int64_t t) -> int64_t {  // label, or mask
            if (t >= p.rows)
                return 0;
            if (kList)
                return p.row_mask != nullptr ? p.row_mask[row_at(t)] : 1;
            return p.labels[row_at(t)];
        };
        int64_t t = cluster;
        int64_t key = key_of(t);
        int64_t n_items = 0;
        uint32_t i = 0, retired = 0;
        const auto retire_below = [&](uint32_t n) {
            while (ok && retired < n)
                retire(retired++);
            return ok;
        };
        for (;; ++i) {
            const int q = i % Q;
            RowSlot &w = slots[q];
            __syncwarp();
            const bool end = t >= p.rows;
            const int64_t r = row_at(t);
            int state = end ? kRowEnd : kRowLive;
            if (!end) {
                if (kList ? key == 0 : key == p.ignore_index || r < lo || r >= hi)
                    state = kRowSkip;
                else if (!kList && (key < 0 || key >= V))
                    state = kRowInvalid;
            }
            const T *row = static_cast<const T *>(p.logits) + r * p.row_stride;
            uint32_t repeated = 0;
            if (lane == 0) {
                w.r = r;
                w.state = w.early = state;
                w.streamed = state == kRowLive;
                w.y = static_cast<int>(key);
                mbar_arrive(&row_bar[q]);
            }
            if (kList && state == kRowLive &&
                list_columns<T, NC>(p, r, slice_of(row), list_of(q), lane, repeated)) {
                state = kRowInvalid;
                if (lane == 0)
                    w.state = w.early = state;
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&cols_bar[q]);
            if (state == kRowInvalid && lane == 0 && split == 0)
                report(p.dev_status, kList ? GBCE_DEV_BAD_INDEX : GBCE_DEV_BAD_LABEL);
            if (i == 0 && p.ticket != nullptr)
                grid_dependency_wait();
            if (i == 0 && kGrad && p.n_items != nullptr && p.reduction == GBCE_MEAN)
                n_items = *p.n_items;
            if (i == 0 && p.n_items_out != nullptr &&
                (blockIdx.x == 0 || (kGrad && p.reduction == GBCE_MEAN))) {
                // one row per CTA at most: every CTA counts the rows that are kept
                for (int64_t j = lane; j < p.rows; j += 32)
                    n_items += kList ? (p.row_mask == nullptr || p.row_mask[j] != 0)
                                     : p.labels[j] != p.ignore_index;
#pragma unroll
                for (int off = 16; off > 0; off >>= 1)
                    n_items += __shfl_xor_sync(0xffffffffu, n_items, off);
                if (blockIdx.x == 0 && lane == 0)
                    *p.n_items_out = n_items;
            }
            if (i == 0 && p.zero_out != nullptr && blockIdx.x == 0 && lane == 0)
                *p.zero_out = 0;
            if (state == kRowLive) {
                // the row's own values, one lane each
                const float *from = nullptr;
                float *to = nullptr;
                if (!kStats && lane < 2) {
                    from = p.rest_state + 2 * r + lane;
                    to = lane == 0 ? &w.m : &w.s;
                }
                if (OP == kOpPolicy && lane >= 2 && lane < 5) {
                    from = lane == 2   ? p.policy.advantages
                           : lane == 3 ? p.policy.old_logp
                                       : p.policy.ref_logp;
                    from = from != nullptr ? from + r : nullptr;
                    to = lane == 2 ? &w.adv : lane == 3 ? &w.old_lp : &w.ref_lp;
                }
                const float value = from != nullptr ? *from : 0.0f;
                float xy = 0.0f, gt = 0.0f;
                if (!kList && lane == 5)
                    xy = E::load(row + key);
                if (kGrad && lane == 6)
                    gt = scaled(post_upstream(p, r, n_items), inv_t);
                if (to != nullptr)
                    *to = value;
                if (!kList && lane == 5)
                    w.xy = xy;
                if (kGrad && lane == 6)
                    w.gt = gt;
                if (kList)
                    list_teacher<T>(p, r, row, list_of(q), w, lane, repeated);
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&list_bar[q]);
            if (end)
                break;
            // The next row is taken once this one is swept (the rows before it are
            // retired): one row ahead hides a list's latency, and with more a CTA could
            // have several rows to go while others have none (two or three further:
            // policy loss, 1922 x 32768 bf16 with a third of the rows live 47 -> 40.5 us,
            // preference loss, 4000 x 20000 98 -> 92 us).
            if (!retire_below(i))
                break;
            t += clusters;
            if (p.ticket != nullptr) {
                int32_t drawn = 0;
                if (lane == 0)
                    drawn = atomicAdd(p.ticket, 1);
                t = clusters + __shfl_sync(0xffffffffu, drawn, 0);
            }
            key = key_of(t);
            if (kList && t < p.rows)
                prefetch_entries(p, row_at(t), lane);
        }
        retire_below(i);
        if (!ok && lane == 0)
            report(p.dev_status, GBCE_DEV_TIMEOUT);
        return;
    }

    // ------------------------------------------------------------ producer
    if (warp == NCW) {
        if (lane != 0)
            return;
        const uint64_t keep = policy_evict_last(), stream = policy_evict_first();
        uint32_t seq = 0, pos = 0, lap = 0;  // chunks issued; ring position and its lap
        bool ok = true;
        for (uint32_t i = 0; ok; ++i) {
            const int q = i % Q;
            if (!mbar_wait(&row_bar[q], (i / Q) & 1)) {
                ok = false;
                break;
            }
            const int64_t r = slots[q].r;
            const bool streamed = slots[q].streamed != 0;
            // (the state that the list warp may change later is not read here)
            const bool end = r >= p.rows || r < 0;
            mbar_arrive(&free_bar[q]);
            if (end)
                break;
            if (!streamed)
                continue;
            const T *row = static_cast<const T *>(p.logits) + r * p.row_stride;
            const Slice sl = slice_of(row);
            const char *body = reinterpret_cast<const char *>(row + sl.g.head) + sl.v0 * 16;
            const int64_t total = (sl.v1 - sl.v0) * 16;
            // gradient rows of another phase need the vector behind each chunk too
            int64_t more = 0;
            if (kGrad &&
                store_geom<T>(static_cast<const T *>(p.dlogits) + r * p.d_stride, sl.g, V).sh != 0)
                more = 16;
            const int64_t total_grad = more != 0 && sl.v1 < sl.g.nvec ? total + 16 : total;
            for (int pass = 0; pass < kPasses && ok; ++pass)
                for (int64_t off = 0; off < total; off += CHUNK, ++seq) {
                    if (lap > 0 && !mbar_wait(&empty_bar[pos], (lap - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    if (kStats)
                        fence_before_refill();
                    const bool grad = kGrad && pass == kPasses - 1;
                    const int64_t left = (grad ? total_grad : total) - off;
                    const int64_t most = CHUNK + (grad ? more : 0);
                    const uint32_t bytes = static_cast<uint32_t>(left < most ? left : most);
                    mbar_arrive_expect_tx(&full_bar[pos], bytes);
                    bulk_load(ring + pos * PITCH, body + off, bytes, &full_bar[pos],
                              pass + 1 < kPasses || r >= p.keep_from ? keep : stream);
                    if (++pos == S) {
                        pos = 0;
                        ++lap;
                    }
                }
        }
        if (!ok)
            report(p.dev_status, GBCE_DEV_TIMEOUT);
        // no copy may still be in flight when the CTA exits
        for (uint32_t j = (seq > S ? seq - S : 0); j < seq; ++j)
            mbar_wait(&full_bar[j % S], (j / S) & 1);
        return;
    }

    // ------------------------------------------------------------ consumers
    uint32_t pos = 0, lap = 0;
    bool alive = true;
    uint32_t swept_rows = 0;
    for (uint32_t i = 0;; ++i) {
        const int q = i % Q;
        if (!mbar_wait(&cols_bar[q], (i / Q) & 1)) {
            report(p.dev_status, GBCE_DEV_TIMEOUT);
            break;
        }
        RowSlot &w = slots[q];
        const int early = w.early;
        if (early == kRowEnd)
            break;
        const int64_t r = w.r;
        const T *row = static_cast<const T *>(p.logits) + r * p.row_stride;
        T *drow = kGrad ? static_cast<T *>(p.dlogits) + r * p.d_stride : nullptr;
        const Slice sl = slice_of(row);
        const int32_t nvec = static_cast<int32_t>(sl.v1 - sl.v0);
        const int32_t nchunks = (nvec + CV - 1) / CV;
        const int32_t head = static_cast<int32_t>(sl.g.head);
        const auto wait_chunk = [&] {
            if (alive && !mbar_wait(&full_bar[pos], lap & 1)) {
                alive = false;
                report(p.dev_status, GBCE_DEV_TIMEOUT);
            }
            return reinterpret_cast<uint4 *>(ring + pos * PITCH);
        };
        const auto done_chunk = [&] {
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&empty_bar[pos]);
            if (++pos == S) {
                pos = 0;
                ++lap;
            }
        };
        // the rest of a row that turns out to be left out or invalid: its copies
        // (of `passes` more passes) are let go by, and its gradient is filled
        const auto drop = [&](int state, int passes, bool swept) {
            for (int32_t j = 0; j < nchunks * passes; ++j) {
                wait_chunk();
                done_chunk();
            }
            if (kStats && !swept && tid == 0)
                mbar_arrive(&stat_bar[q]);  // (every row completes a phase of it)
            if (kGrad) {
                const float fill = state == kRowSkip ? 0.0f : kQuietNan;
                const RowGeom gd = row_geom<T>(drow, V);
                const int64_t d0 = gd.nvec * split / C, d1 = gd.nvec * (split + 1) / C;
                float f[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    f[e] = fill;
                const uint4 pat = E::pack(f);
                uint4 *body = reinterpret_cast<uint4 *>(drow + gd.head);
                for (int64_t v = d0 + tid; v < d1; v += NC)
                    st_cs_v4(body + v, pat);
                if (sl.first && tid < gd.head)
                    E::store(drow + tid, fill);
                if (sl.last && gd.tail0 + tid < V)
                    E::store(drow + gd.tail0 + tid, fill);
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&free_bar[q]);
        };
        if (early != kRowLive) {
            drop(early, w.streamed ? kPasses : 0, false);
            continue;
        }

        const int32_t col0 = head + static_cast<int32_t>(sl.v0) * VEC;  // of the slice's vector 0
        float m, s;
        if (kStats) {
            // the listed columns this thread owns
            const ListRef L = kList ? list_at(lists + q * list_words(NC, static_cast<int>(p.k)), NC,
                                              static_cast<int>(p.k))
                                    : ListRef{};
            const int own = kList ? L.head[tid] : -1;
            int32_t own_col = -1;
            bool own_any = own >= 0, own_more = false;  // one of them, more than one
            if constexpr (kList) {
                if (own_any) {
                    own_col = L.col[own];
                    own_more = L.next[own] >= 0;
                }
            } else if (column_owner<VEC, NC>(sl, w.y) == tid) {
                own_col = w.y;
                own_any = true;
            }
            const auto each_own = [&](auto &&f) {
                f(own_col);
                if constexpr (kList) {
                    if (own_more)
                        for (int j = L.next[own]; j >= 0; j = L.next[j])
                            f(L.col[j]);
                }
            };
            const auto is_listed = [&](int32_t at) {
                bool hit = false;
                each_own([&](int32_t col) { hit |= col == at; });
                return hit;
            };
            RestStats st;
            if (sl.first && tid < sl.g.head)
                st.add1(is_listed(tid) ? kNegInf : E::load(row + tid), c, p.far);
            if (sl.last && sl.g.tail0 + tid < V)
                st.add1(is_listed(static_cast<int32_t>(sl.g.tail0) + tid)
                            ? kNegInf
                            : E::load(row + sl.g.tail0 + tid),
                        c, p.far);
            for (int32_t j = 0; j < nchunks; ++j) {
                uint4 *chunk = wait_chunk();
                const int32_t vb0 = j * CV;
                const int32_t nv = nvec - vb0 < CV ? nvec - vb0 : CV;
                if (own_any && alive) {
                    // listed columns leave the sum: -inf in the copied row, written
                    // by the thread that alone reads their vector
                    each_own([&](int32_t col) {
                        const int32_t e = col - col0 - vb0 * VEC;
                        if (col >= col0 && e >= 0 && e < nv * VEC)
                            reinterpret_cast<T *>(chunk)[e] = neg_inf_as(T());
                    });
                }
                if (alive && nv == CV) {
                    uint4 raw[PER_THREAD];
#pragma unroll
                    for (int u = 0; u < PER_THREAD; ++u)
                        raw[u] = chunk[tid + u * NC];
#pragma unroll
                    for (int u = 0; u < PER_THREAD; u += 2) {
                        const float own = FastVec<T>::vmax(raw[u], raw[u + 1]);
                        // (many warps: the running max rises for the whole warp at once)
                        rest_take<T>(st, raw[u], raw[u + 1],
                                     NCW > 8 ? warp_max_active(own) : own, c, p.far);
                    }
                } else if (alive) {
                    for (int32_t v = tid; v < nv; v += NC)
                        rest_take<T>(st, chunk[v], c, p.far);
                }
                done_chunk();
            }
            // each warp's state, one barrier, then every warp merges them all
            const int rb = static_cast<int>(swept_rows++ & 1u);
            m = st.m;
            s = st.sum();
            if (s != s)  // (a thread that met only NaN has no max: its NaN must still count)
                m = fmaxf(m, 0.0f);
            warp_merge_rest(m, s, c, st.residual(c));
            if (lane == 0) {
                red_m[rb][warp] = m;
                red_s[rb][warp] = s;
            }
            named_sync(1, NC);
            m = lane < NCW ? red_m[rb][lane] : kNegInf;
            s = lane < NCW ? red_s[rb][lane] : 0.0f;
            warp_merge_rest(m, s, c);
            if (C > 1) {
                // the slices' partials, to every CTA of the row
                if (warp == 0) {
                    cluster_wait();  // every peer's mbarriers exist
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&xbar, C * static_cast<uint32_t>(sizeof(float4)));
                        const uint32_t at = smem_addr(&xchg[split]), bar = smem_addr(&xbar);
                        for (int t = 0; t < C; ++t)
                            st_async_v4(map_to_rank(at, t), make_float4(m, s, 0.0f, 0.0f),
                                        map_to_rank(bar, t));
                    }
                    __syncwarp();
                }
                if (!mbar_wait_cluster(&xbar, 0)) {
                    alive = false;
                    report(p.dev_status, GBCE_DEV_TIMEOUT);
                }
                m = kNegInf;
                s = 0.0f;
                for (int t = 0; t < C; ++t)
                    merge_rest(m, s, xchg[t].x, xchg[t].y, c);
            }
            if (tid == 0) {
                w.m = m;
                w.s = s;
                mbar_arrive(&stat_bar[q]);
            }
        }

        if (kGrad) {
            if (!mbar_wait(&list_bar[q], (i / Q) & 1)) {
                report(p.dev_status, GBCE_DEV_TIMEOUT);
                break;
            }
            if (kList && w.state != kRowLive) {
                drop(w.state, 1, true);
                continue;
            }
            if (!kStats) {
                m = w.m;
                s = w.s;
            }
            const float gt = w.gt;
            float gs;
            if (kList) {
                gs = gt * rest_gap(m, s, w.ml, w.sl, w.lp_rest, c, inv_t);
            } else {
                const TokenTerms y = token_terms(m, s, w.xy, inv_t);
                float slope = gt;  // (g / T) dloss / dlog p
                if (OP == kOpPolicy) {
                    float loss, dlp;
                    policy_row(p.policy, w.adv, w.old_lp, w.ref_lp, y.lp, loss, dlp);
                    slope *= dlp;
                }
                gs = -slope * y.other;
            }
            const GradConsts gk = rest_consts<T>(m, s, c.hi + c.lo, gs);
            constexpr int32_t kNoLabel = 0x7fffffff;
            const StoreGeom dg = store_geom<T>(drow, sl.g, V);
            const int sh = dg.sh;
            if (sl.first && tid < dg.begin)
                E::store(drow + tid, grad_scalar(E::load(row + tid), gk));
            if (sl.last && dg.end + tid < V)
                E::store(drow + dg.end + tid, grad_scalar(E::load(row + dg.end + tid), gk));
            const int32_t stored = stored_range<VEC>(sl, dg, V).vecs;
            T *dbase = drow + col0 + sh;
            for (int32_t j = 0; j < nchunks; ++j) {
                const uint4 *chunk = wait_chunk();
                const int32_t vb0 = j * CV;
                const int32_t nv = stored - vb0 < CV ? stored - vb0 : CV;
                T *d = dbase + vb0 * VEC;
                if (alive && nv == CV) {
                    uint4 raw[PER_THREAD];
                    if (sh == 0) {
#pragma unroll
                        for (int u = 0; u < PER_THREAD; ++u)
                            raw[u] = chunk[tid + u * NC];
                    } else {
#pragma unroll
                        for (int u = 0; u < PER_THREAD; ++u)
                            raw[u] = shifted<T>(chunk[tid + u * NC], chunk[tid + u * NC + 1], sh);
                    }
#pragma unroll
                    for (int u = 0; u < PER_THREAD; ++u)
                        st_cs_v4(d + (tid + u * NC) * VEC,
                                 GradVec<T>::run(raw[u], kNoLabel, gk));
                } else if (alive) {
                    for (int32_t v = tid; v < nv; v += NC) {
                        const uint4 raw =
                            sh == 0 ? chunk[v] : shifted<T>(chunk[v], chunk[v + 1], sh);
                        st_cs_v4(d + v * VEC, GradVec<T>::run(raw, kNoLabel, gk));
                    }
                }
                done_chunk();
            }
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&free_bar[q]);
    }
}

// ------------------------------------------------------------------- launches

// Shared memory of an SM, and what a CTA's static arrays and the system take of it.
constexpr int kSmemPerSm = 228 * 1024, kSmemPerCta = 2048 + 1024;
// Bytes of rows that may wait in L2 for their gradient pass, beside the gradients
// of others; where all of them do at once.
constexpr int64_t kPostL2Budget = int64_t(76) << 20, kPostL2Wave = int64_t(88) << 20;
// The least columns a slice of a split row has.
constexpr int64_t kPostSliceElems = 8192;

struct PostLaunch {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    PostLaunch(int64_t ctas, int threads, int smem, int splits, cudaStream_t stream)
    {
        cfg.gridDim = dim3(static_cast<unsigned>(ctas));
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (splits > 1) {
            attr[1].id = cudaLaunchAttributeClusterDimension;
            attr[1].val.clusterDim.x = static_cast<unsigned>(splits);
            attr[1].val.clusterDim.y = 1;
            attr[1].val.clusterDim.z = 1;
            cfg.numAttrs = 2;
        }
    }
};

template <typename T, int OP, int PASS, int SHAPE>
cudaError_t launch_post_shape(const PostParams &params, int sms, cudaStream_t stream)
{
    using Shape = PostShape<SHAPE>;
    static std::atomic<uint64_t> attr_done{0};
    static std::atomic<int> most_clusters[64][kMaxClusterCtas + 1] = {};
    auto kernel = post_kernel<T, OP, PASS, SHAPE>;
    cudaError_t err = ensure_smem_attr(kernel, post_smem<SHAPE>(OP, kMaxListed), attr_done);
    if (err != cudaSuccess)
        return err;
    constexpr int threads = post_threads<SHAPE>();
    const int smem = post_smem<SHAPE>(OP, params.k);
    PostParams p = params;
    const int fit = kSmemPerSm / (smem + kSmemPerCta);
    int64_t slots = static_cast<int64_t>(sms) * (fit < Shape::kCtasPerSm ? fit : Shape::kCtasPerSm);
    if (p.splits > 1) {
        // the largest cluster for which every row's is resident at once (a
        // cluster must fit one GPC); the query runs once per device and size
        int dev = 0;
        if ((err = cudaGetDevice(&dev)) != cudaSuccess)
            return err;
        int C = p.splits;
        for (; C > 1 && dev < 64; --C) {
            int n = most_clusters[dev][C].load(std::memory_order_relaxed);
            if (n == 0) {
                PostLaunch probe(C * p.rows, threads, post_smem<SHAPE>(OP, kMaxListed), C, nullptr);
                probe.cfg.attrs = &probe.attr[1];  // (the cluster alone)
                probe.cfg.numAttrs = 1;
                if (cudaOccupancyMaxActiveClusters(&n, kernel, &probe.cfg) != cudaSuccess || n < 1) {
                    (void)cudaGetLastError();
                    n = -1;  // no answer: no split of this size
                }
                most_clusters[dev][C].store(n, std::memory_order_relaxed);
            }
            if (n >= p.rows)
                break;
        }
        p.splits = C;
    }
    int64_t grid = p.rows * p.splits;
    if (p.splits == 1) {
        if (PASS == kPassFused && SHAPE == kShapeLong) {
            // a row stays in L2 from its first read to its second: fewer CTAs
            // where the rows are long, but not below half the SMs
            const int64_t fit_l2 = kPostL2Budget / (p.vocab * static_cast<int64_t>(sizeof(T)) + 1);
            const int64_t least = sms / 2 > 0 ? sms / 2 : 1;
            if (fit_l2 < slots)
                slots = fit_l2 > least ? fit_l2 : least;
        }
        if (p.rows > slots) {
            // rows beyond the first wave go by ticket: zeroed, and the items
            // counted, by a kernel before this one
            grid = slots;
            if (p.ticket == nullptr)
                err = cudaSuccess;  // (no workspace: a static walk)
            else if (p.n_items_out == nullptr)
                err = cudaMemsetAsync(p.ticket, 0, sizeof(int32_t), stream);
            else if (OP == kOpDistill)
                err = launch_count_mask(p.row_mask, p.rows, p.n_items_out, p.ticket, stream);
            else
                err = launch_count_items(p.labels, p.rows, p.ignore_index, p.n_items_out, p.ticket,
                                         nullptr, nullptr, stream);
            if (err != cudaSuccess)
                return err;
            if (p.n_items_out != nullptr)
                p.n_items = p.n_items_out;
            p.n_items_out = nullptr;
        } else {
            p.ticket = nullptr;
        }
    }
    if (grid == p.rows * p.splits)
        p.ticket = nullptr;
    const PostLaunch l(grid, threads, smem, p.splits, stream);
    err = cudaLaunchKernelEx(&l.cfg, kernel, p);
    note_launches(1);
    return err != cudaSuccess ? err : cudaGetLastError();
}

// The CTA shape for streamed rows (longer than kShortRowBytes) that are not split.
//
// Fused calls re-read each row from L2, so the rows in flight (one per CTA)
// must fit there: of the shapes for which they do, the one with the most CTAs
// for rows of one wave (small CTAs hide a row's serial steps, its list and its
// merge, best), but mid where one wave of those holds the rows and they are
// long; the mid shape's larger ring for several waves.  Measured in us, short /
// mid / long: distillation, 32 entries, 700 x 60000 bf16 39 / 44 / 50, 500 x 32768
// fp32 31 / 38 / 40, 300 x 100000 bf16 33 / 28 / 33, 4096 x 32768 fp32 214 / 179 / 229,
// 8192 x 65536 bf16 422 / 346 / 426, 2000 x 100000 181 / 158 / 150, 4096 x 152064 557 /
// 524 / 412; policy loss, 4000 x 60000 188 / 158 / 197, 2000 x 100000 177 / 156 / 149.
// One pass only (nothing re-read): one wave by the same rule (both sweeps of the
// preference loss, 700 x 100000 bf16 67 / 81 / 77, 400 x 152064 62 / 59 / 69); several
// waves of long rows want fewer and larger CTAs (1000 x 152064 162 / 142 / 137, 4096 x
// 60000 209 / 207 / 231), lists more of them (distillation in two calls, 4096 x
// 152064 596 / 590 / 607, 4096 x 60000 250 / 254 / 376).
template <typename T>
int post_shape(const PostParams &p, int op, int pass, int sms)
{
    const int64_t row = p.vocab * static_cast<int64_t>(sizeof(T));
    const int64_t many = static_cast<int64_t>(sms) * PostShape<kShapeShort>::kCtasPerSm;
    const int64_t some = static_cast<int64_t>(sms) * PostShape<kShapeMid>::kCtasPerSm;
    const bool one_wave = p.rows <= many, fused = pass == kPassFused;
    if (one_wave && (!fused || p.rows * row <= kPostL2Wave))
        return p.rows <= some && row >= 160 * 1024 ? kShapeMid : kShapeShort;
    if (fused)
        return (p.rows < some ? p.rows : some) * row <= kPostL2Budget ? kShapeMid : kShapeLong;
    if (op == kOpDistill)
        return pass == kPassFwd && row >= 256 * 1024 && p.rows < 4 * some ? kShapeLong : kShapeMid;
    return row < 128 * 1024 ? kShapeMid : kShapeLong;
}

template <typename T, int OP, int PASS>
cudaError_t launch_post_as(PostParams p, cudaStream_t stream)
{
    const int sms = device_sm_count();
    if (sms <= 0)
        return cudaErrorInvalidDevice;
    p.splits = 1;
    // few rows: each one's slices on the CTAs of a cluster
    const int64_t slots = static_cast<int64_t>(sms) * PostShape<kShapeMid>::kCtasPerSm;
    if (p.rows * 2 <= slots && p.vocab >= 2 * kPostSliceElems) {
        int64_t n = slots / p.rows;
        if (n > p.vocab / kPostSliceElems)
            n = p.vocab / kPostSliceElems;
        p.splits = static_cast<int>(n < kMaxClusterCtas ? n : kMaxClusterCtas);
        return launch_post_shape<T, OP, PASS, kShapeMid>(p, sms, stream);
    }
    switch (post_shape<T>(p, OP, PASS, sms)) {
    case kShapeLong:
        return launch_post_shape<T, OP, PASS, kShapeLong>(p, sms, stream);
    case kShapeMid:
        return launch_post_shape<T, OP, PASS, kShapeMid>(p, sms, stream);
    default:
        return launch_post_shape<T, OP, PASS, kShapeShort>(p, sms, stream);
    }
}

template <typename T>
cudaError_t launch_post(const PostParams &p, int op, int pass, cudaStream_t stream)
{
    if (p.rows == 0)
        return cudaSuccess;
    // Short rows are kept in shared memory; a few that would make a CTA long are
    // split over a cluster below (policy loss, 8 x 50000 bf16 7.9 us, whole 8.5; 100 x
    // 40000 11.8, whole 8.9; 24 x 16384 6.9, whole 6.3).
    const int64_t row = p.vocab * static_cast<int64_t>(sizeof(T));
    if (row <= kShortRowBytes && (row <= kShortAlwaysBytes || p.rows > kShortFewest))
        return launch_post_short<T>(p, op, pass, stream);
    if (op == kOpPolicy)
        return launch_post_as<T, kOpPolicy, kPassFused>(p, stream);
    if (op == kOpToken)
        return pass == kPassFwd ? launch_post_as<T, kOpToken, kPassFwd>(p, stream)
                                : launch_post_as<T, kOpToken, kPassBwd>(p, stream);
    if (pass == kPassFwd)
        return launch_post_as<T, kOpDistill, kPassFwd>(p, stream);
    if (pass == kPassBwd)
        return launch_post_as<T, kOpDistill, kPassBwd>(p, stream);
    return launch_post_as<T, kOpDistill, kPassFused>(p, stream);
}

}  // namespace gbce
