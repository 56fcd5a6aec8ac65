// Row kernels of the post-training losses over [rows, vocab] logits (sm_103a):
// distillation from a teacher's top logits, and the clipped policy loss.
//
// Both losses see a row as a few LISTED columns (the teacher's entries; the
// sampled token) and the REST.  One sweep takes the online (max m, sum s) of
// the rest with the listed columns left out; the listed logits are gathered on
// the side, so that 1 - p never comes from a difference with 1 (the form of
// the cross-entropy kernels).  The loss and every gradient then follow from
// (m, s) and the listed logits:
//   unlisted j:  dx_j = gs 2^{(x_j - m) c - log2 s}, gs = (g / T) times the
//                rest's whole share of the gradient,
//   listed k:    a value of its own, stored over the sweep's by the thread
//                that owns the column's vector.
#pragma once

#include "gbce_kernels.cuh"
#include "gbce_post.h"

namespace gbce {

constexpr float kQuietNan = __builtin_nanf("");

// ------------------------------------------------------------ listed columns

// The listed columns of one row, in shared memory.  Column col of a row is
// owned by one consumer thread (the one whose sweep reads it); the entries of
// an owner form a chain head[owner] -> next -> ... of which a thread walks only
// its own, so the sweep and the patches need no barrier between threads.
template <int NC>
struct ListBuf {
    int32_t col[kMaxListed];  // column; -1: no entry (or a repeat of an earlier one)
    float x[kMaxListed];      // student logit
    float lp[kMaxListed];     // teacher's log p
    int32_t next[kMaxListed];
    int32_t head[NC];
    float ml, sl;   // listed logits: max, and sum of 2^{(x - ml) c} without one holder of the max
    float lp_rest;  // teacher's log p of the unlisted columns (-inf: none)
    int state;      // RowState
};

enum RowState : int {
    kRowLive = 0,
    kRowSkip = 1,     // left out, or a teacher without mass: loss 0, gradient 0
    kRowInvalid = 2,  // NaN outputs (a bad index or label, a NaN teacher logit)
};

// Which slice of a row a CTA sweeps, and which of its threads owns a column.
struct Slice {
    RowGeom g;
    int64_t v0, v1;  // body vectors of the slice
    bool first, last;  // the slice holds the row's scalar head / tail
};

template <int VEC, int NC>
__device__ __forceinline__ int column_owner(const Slice &sl, int32_t col)
{
    if (col < sl.g.head)
        return col;
    if (col >= sl.g.tail0)
        return static_cast<int>(col - sl.g.tail0);
    const int64_t v = (col - sl.g.head) / VEC - sl.v0;
    return static_cast<int>((v % NC + NC) % NC);
}

// Whether the slice sweeps this column.
template <int VEC>
__device__ __forceinline__ bool in_slice(const Slice &sl, int32_t col)
{
    if (col < sl.g.head)
        return sl.first;
    if (col >= sl.g.tail0)
        return sl.last;
    const int64_t v = (col - sl.g.head) / VEC;
    return v >= sl.v0 && v < sl.v1;
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

// Read the teacher's entries of row r into L (one warp).  An index listed
// twice is one column with the sum of both probabilities.  The teacher's
// distribution is the softmax over its logits / T and teacher_rest.
template <typename T, int NC>
__device__ void build_list(const PostParams &p, int64_t r, const T *row, const Slice &sl,
                           ListBuf<NC> &L, int lane)
{
    constexpr int VEC = Elem<T>::kVec;
    constexpr int kPer = kMaxListed / 32;
    const int K = static_cast<int>(p.k);
    const float c = p.c;
    const float rest = p.teacher_rest != nullptr ? p.teacher_rest[r] : kNegInf;
    bool bad = false, nan_t = !(rest < __builtin_huge_valf());
    for (int i = lane; i < NC; i += 32)
        L.head[i] = -1;
    for (int k = lane; k < K; k += 32) {
        const int64_t t = p.index[r * K + k];
        const bool here = t >= 0 && t < p.vocab;
        bad |= !here && t != -1;
        float tau = kNegInf, x = kNegInf;
        if (here) {
            tau = p.teacher[r * K + k] / p.T;
            x = Elem<T>::load(row + t);
            nan_t |= !(tau < __builtin_huge_valf());
        }
        L.col[k] = here ? static_cast<int32_t>(t) : -1;
        L.x[k] = x;
        L.lp[k] = tau;
    }
    bad = __any_sync(0xffffffffu, bad);
    nan_t = __any_sync(0xffffffffu, nan_t);
    __syncwarp();
    for (int k = lane; k < K; k += 32)
        if (L.col[k] >= 0)
            L.next[k] = atomicExch(&L.head[column_owner<VEC, NC>(sl, L.col[k])], k);
    __syncwarp();
    // repeats: equal columns share an owner, so its chain shows them all
    uint32_t repeat = 0, repeated = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int k = lane + 32 * i;
        if (k >= K || L.col[k] < 0)
            continue;
        for (int j = L.head[column_owner<VEC, NC>(sl, L.col[k])]; j >= 0; j = L.next[j]) {
            if (j != k && L.col[j] == L.col[k])
                (j < k ? repeat : repeated) |= 1u << i;
        }
    }
    // the first of several takes their sum, in entry order
    float tsum[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int k = lane + 32 * i;
        tsum[i] = k < K ? L.lp[k] : kNegInf;
        if ((repeated >> i & 1u) && !(repeat >> i & 1u)) {
            float m = kNegInf, s = 0.0f;
            for (int j = k; j < K; ++j)
                if (L.col[j] == L.col[k])
                    m = fmaxf(m, L.lp[j]);
            for (int j = k; j < K; ++j)
                if (L.col[j] == L.col[k] && L.lp[j] != kNegInf)
                    s += expf(L.lp[j] - m);
            tsum[i] = s > 0.0f ? m + logf(s) : kNegInf;
        }
    }
    __syncwarp();
    // maxima: the teacher's over the entries and the rest, the student's
    float mt = kNegInf, ml = kNegInf;
    int32_t at = INT32_MAX, al = INT32_MAX;
    bool nan_x = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int k = lane + 32 * i;
        if (k >= K || L.col[k] < 0)
            continue;
        if (repeat >> i & 1u) {
            L.col[k] = -1;
            continue;
        }
        L.lp[k] = tsum[i];
        if (tsum[i] > mt) {
            mt = tsum[i];
            at = k;
        }
        const float x = L.x[k];
        nan_x |= x != x || x == __builtin_huge_valf();
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
    float st = (at != -1 && rest != kNegInf) ? expf(rest - mt) : 0.0f, sx = 0.0f;
    st = lane == 0 ? st : 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int k = lane + 32 * i;
        if (k >= K || L.col[k] < 0)
            continue;
        if (k != at && L.lp[k] != kNegInf)
            st += expf(L.lp[k] - mt);
        if (k != al && L.x[k] != kNegInf)
            sx += ex2((L.x[k] - ml) * c);
    }
    st = warp_sum(st);
    sx = warp_sum(sx);
    const float lt = log1pf(st);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int k = lane + 32 * i;
        if (k < K && L.col[k] >= 0)
            L.lp[k] = (L.lp[k] - mt) - lt;
    }
    if (lane == 0) {
        // a row with a NaN (or +inf) listed logit has no softmax
        L.ml = nan_x ? 0.0f : ml;
        L.sl = nan_x ? kQuietNan : sx;
        L.lp_rest = rest == kNegInf ? kNegInf : (rest - mt) - lt;
        L.state = (bad || nan_t) ? kRowInvalid : (mt == kNegInf ? kRowSkip : kRowLive);
    }
    if (bad && lane == 0 && sl.first)
        report(p.dev_status, GBCE_DEV_BAD_INDEX);
}

// ------------------------------------------------------- distillation of a row

// The student's softmax from the rest's state (m, s) and the listed logits'
// (ml, sl): log q_k = (x_k - M) / T - log_s, and log q of the rest.
struct StudentRow {
    float M, log_s, log_rest;
};

__device__ __forceinline__ StudentRow student_row(float m, float s, float ml, float sl, float c,
                                                  float T)
{
    StudentRow q;
    q.M = fmaxf(m, ml);
    const float rest = m == kNegInf ? s : s * ex2((m - q.M) * c);
    const float listed = ml == kNegInf ? 0.0f : (1.0f + sl) * ex2((ml - q.M) * c);
    // log of the whole sum: past its own largest term where that is listed
    q.log_s = ml >= m ? log1pf(sl + rest) : logf(rest + listed);
    // log of the rest's share, by whichever of the two does not cancel
    q.log_rest = rest >= listed ? -log1pf(listed / rest)
                                : (s > 0.0f ? (logf(s) + (m - q.M) / T) - q.log_s : kNegInf);
    if (q.M == kNegInf || listed != listed || rest != rest) {
        q.log_s = kQuietNan;
        q.log_rest = kQuietNan;
    }
    return q;
}

// p phi(u), u = log q - log p, phi(u) = e^u - 1 - u >= 0: one term of
// KL = sum p (log p - log q) written as a sum of non-negative terms (both
// distributions sum to 1, so the extra q - p sum to 0).  A near-converged
// student keeps its loss, where the plain terms cancel to fp32's rounding.
__device__ __forceinline__ float kl_term(float lp, float lq)
{
    const float q = expf(lq);
    if (lp == kNegInf)
        return q;
    const float p = expf(lp), u = lq - lp;
    if (fabsf(u) < 0.25f) {
        // u^2 / 2 + u^3 / 6 + ...: the next term is below 2^-24 of the sum
        float h = 1.0f / 5040.0f;
        h = fmaf(h, u, 1.0f / 720.0f);
        h = fmaf(h, u, 1.0f / 120.0f);
        h = fmaf(h, u, 1.0f / 24.0f);
        h = fmaf(h, u, 1.0f / 6.0f);
        h = fmaf(h, u, 0.5f);
        return p * u * u * h;
    }
    if (u > 1.0f)
        return (q - p) - p * u;
    return p > 0.0f ? p * (expm1f(u) - u) : 0.0f;
}

// q - p without the cancellation of two nearly equal values.
__device__ __forceinline__ float share_gap(float lp, float lq)
{
    if (lp == kNegInf)
        return expf(lq);
    const float u = lq - lp;
    return fabsf(u) < 1.0f ? expf(lp) * expm1f(u) : expf(lq) - expf(lp);
}

// ---------------------------------------------------------- policy of a row

// The clipped policy loss of one row from its log p, and its derivative:
//   rho = e^{lp - old},  loss = -min(rho A, clip(rho) A) + beta (e^d - 1 - d),
//   d = ref - lp;  d loss / d lp = -rho A [not clipped] - beta (e^d - 1).
// At a clip's border the unclipped side is taken.
__device__ __forceinline__ void policy_row(const PolicyTerms &t, int64_t r, float lp, float &loss,
                                           float &dlp)
{
    const float A = t.advantages[r];
    loss = dlp = lp != lp ? kQuietNan : 0.0f;
    if (A != 0.0f && lp == lp) {  // (no advantage: no surrogate, however large the ratio)
        const float rho = t.old_logp != nullptr ? expf(lp - t.old_logp[r]) : 1.0f;
        const float edge = A > 0.0f ? 1.0f + t.clip_high : 1.0f - t.clip_low;
        const bool held = A > 0.0f ? rho > edge : rho < edge;
        loss = -A * (held ? edge : rho);
        dlp = held ? 0.0f : -A * rho;
        if (rho != rho || A != A)
            loss = dlp = kQuietNan;
    }
    if (t.ref_logp != nullptr && t.kl_beta != 0.0f) {
        const float d = t.ref_logp[r] - lp, e = expm1f(d);
        float k3 = e - d;
        if (fabsf(d) < 0.25f) {
            float h = 1.0f / 5040.0f;
            h = fmaf(h, d, 1.0f / 720.0f);
            h = fmaf(h, d, 1.0f / 120.0f);
            h = fmaf(h, d, 1.0f / 24.0f);
            h = fmaf(h, d, 1.0f / 6.0f);
            h = fmaf(h, d, 0.5f);
            k3 = d * d * h;
        }
        loss = fmaf(t.kl_beta, k3, loss);
        dlp = fmaf(-t.kl_beta, e, dlp);
    }
}

// ------------------------------------------------------------- the gradient

// Constants of the sweep over the unlisted columns: gs 2^{(x - m) c - log2 s}.
// Every exponent is <= 0 and relative to the rest's own max, so no element
// carries the rounding of a large offset.
__device__ __forceinline__ GradConsts rest_consts(float m, float s, float c, float gs)
{
    const bool none = !(s > 0.0f) || !isfinite(m);  // nothing unlisted has mass
    GradConsts k;
    k.c = c;
    k.off = 0.0f;
    k.nxy = none ? 0.0f : -m;
    k.kb = none ? 0.0f : -log2f(s);
    k.kbx = none ? 0.0f : fmaf(-m, c, k.kb);
    k.gs = none && !(s != s) && m != __builtin_huge_valf() ? 0.0f : gs;
    k.dy = 0.0f;
    k.c0 = 0.0f;
    k.ea = k.eb = 0.0f;
    return k;
}

__device__ __forceinline__ float post_upstream(const PostParams &p, int64_t r)
{
    if (p.reduction == 0)
        return p.grad_out[r];
    if (p.reduction == 1)
        return p.grad_out[0];
    const int64_t n = *p.n_items;
    return n > 0 ? p.grad_out[0] / static_cast<float>(n) : 0.0f;
}

// ------------------------------------------------------------ the row kernel

constexpr int kPostWarps = 8;

// One CTA per row: warp 0 gathers the listed columns, every thread sweeps its
// vectors of the row for (m, s), and sweeps them again for the gradient.
template <typename T, int OP, int PASS>
__global__ void __launch_bounds__(kPostWarps * 32) post_row_kernel(const PostParams p)
{
    using E = Elem<T>;
    constexpr int VEC = E::kVec;
    constexpr int NCW = kPostWarps, NC = NCW * 32;
    __shared__ ListBuf<NC> L;
    __shared__ float red_m[NCW], red_s[NCW];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t r = blockIdx.x, V = p.vocab;
    const T *row = static_cast<const T *>(p.logits) + r * p.row_stride;
    T *drow = PASS == kPassFwd ? nullptr : static_cast<T *>(p.dlogits) + r * p.d_stride;
    const float c = p.c;

    int state = kRowLive;
    int32_t y = -1;
    if (OP == kOpPolicy) {
        const int64_t lab = p.labels[r];
        state = lab == p.ignore_index ? kRowSkip : (lab < 0 || lab >= V ? kRowInvalid : kRowLive);
        y = state == kRowLive ? static_cast<int32_t>(lab) : -1;
        if (state == kRowInvalid && tid == 0)
            report(p.dev_status, GBCE_DEV_BAD_LABEL);
    } else if (p.row_mask != nullptr && p.row_mask[r] == 0) {
        state = kRowSkip;
    }
    const RowGeom g = row_geom<T>(row, V);
    const Slice sl = {g, 0, g.nvec, true, true};
    if (OP == kOpDistill && state == kRowLive) {
        if (warp == 0)
            build_list<T, NC>(p, r, row, sl, L, lane);
        __syncthreads();
        state = L.state;
    }
    if (state != kRowLive) {
        const float fill = state == kRowSkip ? 0.0f : kQuietNan;
        if (tid == 0) {
            if (PASS != kPassBwd)
                p.loss_rows[r] = fill;
            if (OP == kOpPolicy && p.logp_out != nullptr)
                p.logp_out[r] = fill;
            if (OP == kOpDistill && p.rest_state_out != nullptr) {
                p.rest_state_out[2 * r] = kNegInf;
                p.rest_state_out[2 * r + 1] = 0.0f;
            }
        }
        if (PASS != kPassFwd)
            fill_row_slice<T>(drow, V, 0, 1, fill);
        return;
    }

    // whether this thread's column col is listed
    const auto listed = [&](int32_t col) {
        if (OP == kOpPolicy)
            return col == y;
        for (int j = L.head[tid]; j >= 0; j = L.next[j])
            if (L.col[j] == col)
                return true;
        return false;
    };
    float m, s;
    if (PASS == kPassBwd) {
        m = p.rest_state[2 * r];
        s = p.rest_state[2 * r + 1];
    } else {
        OnlineStats<false> st;
        for_each_own_column<T>(row, g, V, tid, NC, [&](float x, int64_t col) {
            st.add1(listed(static_cast<int32_t>(col)) ? kNegInf : x, c);
        });
        float h = 0.0f;
        m = st.m;
        s = st.sum();
        if (s != s)  // (a thread that met only NaN has no max: its NaN must still count)
            m = fmaxf(m, 0.0f);
        warp_merge_state<kHNone>(m, s, h, c, st.residual(c));
        if (lane == 0) {
            red_m[warp] = m;
            red_s[warp] = s;
        }
        __syncthreads();
        m = lane < NCW ? red_m[lane] : kNegInf;
        s = lane < NCW ? red_s[lane] : 0.0f;
        warp_merge_state<kHNone>(m, s, h, c);
    }

    float gs = 0.0f, gt = 0.0f;  // the rest's share of the gradient; g / T
    float dy = 0.0f;             // policy: the gradient at the label
    StudentRow q;
    if (OP == kOpPolicy) {
        const float lp = finalize_logp(m, s, E::load(row + y), p.T);
        float loss, dlp;
        policy_row(p.policy, r, lp, loss, dlp);
        if (tid == 0) {
            p.loss_rows[r] = loss;
            if (p.logp_out != nullptr)
                p.logp_out[r] = lp;
        }
        dy = -(post_upstream(p, r) / p.T * dlp) * expm1f(lp);
        gs = -dy;
    } else {
        q = student_row(m, s, L.ml, L.sl, c, p.T);
        if (PASS != kPassBwd && warp == 0) {
            float kl = lane == 0 ? kl_term(L.lp_rest, q.log_rest) : 0.0f;
            for (int k = lane; k < p.k; k += 32)
                if (L.col[k] >= 0)
                    kl += kl_term(L.lp[k], (L.x[k] - q.M) / p.T - q.log_s);
            kl = warp_sum(kl);
            if (lane == 0) {
                p.loss_rows[r] = kl;
                if (p.rest_state_out != nullptr) {
                    p.rest_state_out[2 * r] = m;
                    p.rest_state_out[2 * r + 1] = s;
                }
            }
        }
        if (PASS != kPassFwd) {
            gt = post_upstream(p, r) / p.T;
            gs = gt * share_gap(L.lp_rest, q.log_rest);
        }
    }
    if (PASS == kPassFwd)
        return;

    const GradConsts gk = rest_consts(m, s, c, gs);
    for (int64_t e = tid; e < g.head; e += NC)
        E::store(drow + e, grad_scalar(E::load(row + e), gk));
    for (int64_t e = g.tail0 + tid; e < V; e += NC)
        E::store(drow + e, grad_scalar(E::load(row + e), gk));
    const uint4 *body = reinterpret_cast<const uint4 *>(row + g.head);
    constexpr int32_t kNoLabel = 0x7fffffff;
    for (int64_t v = tid; v < g.nvec; v += NC) {
        const uint4 raw = body[v];
        T *d = drow + g.head + v * VEC;
        if (p.vec_store) {
            st_cs_v4(d, GradVec<T>::run(raw, kNoLabel, gk));
        } else {
            float f[VEC];
            GradVec<T>::run_unpacked(raw, kNoLabel, gk, f);
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                E::store(d + e, f[e]);
        }
    }
    // the listed columns, over this thread's own stores
    if (OP == kOpPolicy) {
        if (column_owner<VEC, NC>(sl, y) == tid)
            E::store(drow + y, dy);
    } else {
        for (int j = L.head[tid]; j >= 0; j = L.next[j])
            if (L.col[j] >= 0)
                E::store(drow + L.col[j],
                         gt * share_gap(L.lp[j], (L.x[j] - q.M) / p.T - q.log_s));
    }
}

template <typename T, int OP, int PASS>
cudaError_t launch_post_as(const PostParams &p, cudaStream_t stream)
{
    post_row_kernel<T, OP, PASS>
        <<<static_cast<unsigned>(p.rows), kPostWarps * 32, 0, stream>>>(p);
    note_launches(1);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_post(const PostParams &p, int op, int pass, cudaStream_t stream)
{
    if (p.rows == 0)
        return cudaSuccess;
    if (op == kOpPolicy)
        return launch_post_as<T, kOpPolicy, kPassFused>(p, stream);
    if (pass == kPassFwd)
        return launch_post_as<T, kOpDistill, kPassFwd>(p, stream);
    if (pass == kPassBwd)
        return launch_post_as<T, kOpDistill, kPassBwd>(p, stream);
    return launch_post_as<T, kOpDistill, kPassFused>(p, stream);
}

}  // namespace gbce
