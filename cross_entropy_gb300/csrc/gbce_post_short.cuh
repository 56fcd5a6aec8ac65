// Row kernel of the post-training losses for short rows (sm_103a): a row is
// copied into shared memory whole and both of its sweeps read it there.
//
// The streaming kernel (gbce_post.cuh) spends some 4 to 6 us of one CTA on the
// chain ticket - label - list - merge of every row, which long rows hide and
// short ones do not (policy loss of 8192 rows of 300 bf16 logits: 70 us for 10
// MB).  Here every row has a group of W warps of its own, no row waits for
// another, and the warps of an SM hide each other's chains.  The formulas, the
// states and what is done with bad input are the streaming kernel's.
#pragma once

#include "gbce_post.cuh"

namespace gbce {

// A group takes one row: a warp (four of them in a CTA), or the whole CTA.
template <int W> struct RowGroup {
    static constexpr int kThreads = 32 * W, kRows = W == 1 ? 4 : 1;
    static constexpr int kCta = kThreads * kRows;
    static constexpr int kEntries = (kMaxListed + kThreads - 1) / kThreads;  // of a thread

    __device__ static __forceinline__ void sync()
    {
        if (W == 1)
            __syncwarp();
        else
            __syncthreads();
    }
    // (also a sync())
    __device__ static __forceinline__ bool any(bool x)
    {
        if (W > 1)
            return __syncthreads_or(x);
        __syncwarp();
        return __any_sync(0xffffffffu, x);
    }
};

// Shared memory of a row: its vectors, which begin and end as it lies in memory,
// and the columns and logits of the teacher's entries.
template <typename T> __host__ __device__ __forceinline__ int short_row_bytes(int64_t vocab)
{
    constexpr int VEC = Elem<T>::kVec;
    return static_cast<int>((vocab + 2 * (VEC - 1) + VEC - 1) / VEC) * 16;
}

template <typename T, int W>
__host__ __device__ __forceinline__ int short_smem(int64_t vocab, int op, int64_t k)
{
    const int list = op == kOpDistill ? 8 * ((static_cast<int>(k) + 1) & ~1) : 0;
    return RowGroup<W>::kRows * (short_row_bytes<T>(vocab) + list);
}

// A sum that is led by its largest term: base^m (1 + s), nothing where m is
// -inf.  The largest term stays out of s, so that log1p(s) keeps what the others
// weigh however little that is.
struct LedSum {
    float m, s;

    template <typename Exp> __device__ __forceinline__ void merge(float m2, float s2, Exp exp_of)
    {
        const bool up = m2 > m;
        const float low = up ? m : m2, rest = up ? s : s2;
        const float lead = up ? m2 : m;
        s = up ? s2 : s;
        if (low != kNegInf)
            s += (1.0f + rest) * exp_of(low - lead);
        m = lead;
    }
    // of the warp's lanes, on every lane, in a fixed order
    template <typename Exp> __device__ __forceinline__ void warp_merge(Exp exp_of)
    {
        float M;
        asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(M) : "f"(m));
        const int holder = __ffs(__ballot_sync(0xffffffffu, m == M)) - 1;
        float v = s;
        if ((threadIdx.x & 31) != holder)
            v = m == kNegInf ? 0.0f : (1.0f + s) * exp_of(m - M);
        s = warp_sum(v);
        m = M;
    }
};

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float tag_as(float, int k) { return __int_as_float(k); }
__device__ __forceinline__ __nv_bfloat16 tag_as(__nv_bfloat16, int k)
{
    return __ushort_as_bfloat16(static_cast<unsigned short>(k));
}
__device__ __forceinline__ int tag_of(float x) { return __float_as_int(x); }
__device__ __forceinline__ int tag_of(__nv_bfloat16 x) { return __bfloat16_as_ushort(x); }

// What the warps of a group tell each other after the first sweep.
struct ShortPartial {
    float m, s, teacher_m, teacher_s, student_m, student_s;
    int nans;  // 1: the teacher's, 2: the student's listed logits
};

template <typename T, int OP, int PASS, int W>
__global__ void __launch_bounds__(RowGroup<W>::kCta, W == 8 ? 4 : 8)
    post_short_kernel(const PostParams p, int ordered)
{
    using E = Elem<T>;
    using G = RowGroup<W>;
    constexpr int VEC = E::kVec, NT = G::kThreads, KE = G::kEntries;
    constexpr bool kStats = PASS != kPassBwd, kGrad = PASS != kPassFwd;
    constexpr bool kList = OP == kOpDistill;

    extern __shared__ __align__(128) uint8_t dyn_smem[];
    __shared__ uint64_t copy_bar[G::kRows];
    __shared__ ShortPartial partial[W];
    // each warp's part of the loss, beside `partial`: a slower warp may still be
    // reading that (no barrier lies between the two in the forward pass)
    __shared__ float partial_kl[W];
    __shared__ int64_t counts[G::kCta / 32];

    const int lane = threadIdx.x & 31;
    const int group = W == 1 ? threadIdx.x >> 5 : 0;
    const int tid = W == 1 ? lane : threadIdx.x;  // in the group
    const int warp = W == 1 ? 0 : threadIdx.x >> 5;
    const int64_t V = p.vocab;
    const int K = kList ? static_cast<int>(p.k) : 0;
    const TwoFloat c = {p.c_hi, p.c_lo}, inv_t = {p.it_hi, p.it_lo};
    uint8_t *mine = dyn_smem + group * (short_smem<T, W>(V, OP, p.k) / G::kRows);
    T *buf = reinterpret_cast<T *>(mine);
    int32_t *list_col = reinterpret_cast<int32_t *>(mine + short_row_bytes<T>(V));
    float *list_tau = reinterpret_cast<float *>(list_col + K);

    // With `ordered` the kernel before this one is the library's own count of the
    // rows, which starts once everything before it is complete: only what it wrote
    // is waited for (wait_for_count).
    if (!ordered)
        grid_dependency_wait();
    const int64_t at = static_cast<int64_t>(blockIdx.x) * G::kRows + group;
    const bool inside = at < p.rows;
    const int64_t r = inside ? (p.reverse ? p.rows - 1 - at : at) : 0;
    const T *row = static_cast<const T *>(p.logits) + r * p.row_stride;
    T *drow = kGrad ? static_cast<T *>(p.dlogits) + r * p.d_stride : nullptr;

    // everything that the row needs from elsewhere, asked for at once
    int state = kRowLive, y = 0;
    int64_t key = 1;
    if (inside)
        key = kList ? (p.row_mask != nullptr ? p.row_mask[r] : 1) : p.labels[r];
    int64_t idx[KE];
    float tau[KE], x[KE];
    float rest = kNegInf;
    if constexpr (kList) {
#pragma unroll
        for (int b = 0; b < KE; ++b) {
            const int k = tid + b * NT;
            const bool here = inside && k < K;
            idx[b] = here ? __ldg(p.index + r * K + k) : -1;
            tau[b] = here ? __ldg(p.teacher + r * K + k) : kNegInf;
            x[b] = kNegInf;
        }
        if (inside && p.teacher_rest != nullptr)
            rest = p.teacher_rest[r];
    }
    float adv = 0.0f, old_lp = 0.0f, ref_lp = 0.0f;
    if (OP == kOpPolicy && inside) {
        adv = p.policy.advantages[r];
        old_lp = p.policy.old_logp != nullptr ? p.policy.old_logp[r] : 0.0f;
        ref_lp = p.policy.ref_logp != nullptr ? p.policy.ref_logp[r] : 0.0f;
    }
    float m = kNegInf, s = 0.0f;
    if (!kStats && inside) {
        m = p.rest_state[2 * r];
        s = p.rest_state[2 * r + 1];
    }
    if constexpr (kList) {
        if (key == 0)
            state = kRowSkip;
    } else {
        const int64_t lo = p.row_range != nullptr ? p.row_range[0] : 0;
        const int64_t hi = p.row_range != nullptr ? p.row_range[p.row_range_end] : p.rows;
        if (key == p.ignore_index || r < lo || r >= hi)
            state = kRowSkip;
        else if (key < 0 || key >= V)
            state = kRowInvalid;
        else
            y = static_cast<int>(key);
    }

    const RowGeom g = row_geom<T>(row, V);
    const int phase = static_cast<int>(
        (reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));  // column j is buf[phase + j]
    const int nv = static_cast<int>((phase + V + VEC - 1) / VEC);
    if (inside && state == kRowLive) {
        if (tid == 0) {
            mbar_init(&copy_bar[group], 1);
            fence_barrier_init();
            const uint32_t bytes = static_cast<uint32_t>(g.nvec) * 16u;
            mbar_arrive_expect_tx(&copy_bar[group], bytes);
            if (bytes > 0)
                bulk_load(buf + phase + g.head, row + g.head, bytes, &copy_bar[group],
                          PASS == kPassFwd && r >= p.keep_from ? policy_evict_last()
                                                               : policy_evict_first());
        }
        // the ragged ends, and -inf in the vectors around them
        if (tid < g.head)
            buf[phase + tid] = row[tid];
        if (g.tail0 + tid < V)
            buf[phase + g.tail0 + tid] = row[g.tail0 + tid];
        if (tid < phase)
            buf[tid] = neg_inf_as(T());
        if (phase + V + tid < static_cast<int64_t>(nv) * VEC)
            buf[phase + V + tid] = neg_inf_as(T());
    }
    if (p.zero_out != nullptr && blockIdx.x == 0 && threadIdx.x == 0)
        *p.zero_out = 0;

    int64_t n_items = 0;
    if (p.n_items_out != nullptr &&
        (blockIdx.x == 0 ||
         (kGrad && p.reduction == GBCE_MEAN && (G::kRows > 1 || state == kRowLive)))) {
        // few rows: every CTA that needs it counts the rows that are kept
#pragma unroll 4
        for (int64_t j = threadIdx.x; j < p.rows; j += G::kCta)
            n_items += kList ? (p.row_mask == nullptr || p.row_mask[j] != 0)
                             : p.labels[j] != p.ignore_index;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            n_items += __shfl_xor_sync(0xffffffffu, n_items, off);
        if (lane == 0)
            counts[threadIdx.x >> 5] = n_items;
        __syncthreads();
        n_items = 0;
#pragma unroll
        for (int w = 0; w < G::kCta / 32; ++w)
            n_items += counts[w];
        if (blockIdx.x == 0 && threadIdx.x == 0)
            *p.n_items_out = n_items;
    }
    if (!inside)
        return;
    // (on every way out: the kernel after this one may read the count)
    const auto wait_for_count = [&] {
        if (ordered)
            grid_dependency_wait();
    };

    // a row that is left out or invalid: its outputs
    const auto fill = [&] {
        wait_for_count();
        const float v = state == kRowSkip ? 0.0f : kQuietNan;
        if (kStats && tid == 0) {
            if (p.loss_rows != nullptr)
                p.loss_rows[r] = v;
            if (p.logp_out != nullptr)
                p.logp_out[r] = v;
            if (p.rest_state_out != nullptr) {
                p.rest_state_out[2 * r] = kNegInf;
                p.rest_state_out[2 * r + 1] = 0.0f;
            }
        }
        if (kGrad) {
            const RowGeom gd = row_geom<T>(drow, V);
            float f[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                f[e] = v;
            const uint4 pat = E::pack(f);
            uint4 *body = reinterpret_cast<uint4 *>(drow + gd.head);
            for (int64_t i = tid; i < gd.nvec; i += NT)
                st_cs_v4(body + i, pat);
            if (tid < gd.head)
                E::store(drow + tid, v);
            if (gd.tail0 + tid < V)
                E::store(drow + gd.tail0 + tid, v);
        }
    };
    if (state != kRowLive) {
        if (state == kRowInvalid && tid == 0)
            report(p.dev_status, GBCE_DEV_BAD_LABEL);
        fill();
        return;
    }

    // the copied row, and whether an index is out of range
    bool bad = false;
    int32_t col[KE];
    if constexpr (kList) {
#pragma unroll
        for (int b = 0; b < KE; ++b) {
            const bool here = idx[b] >= 0 && idx[b] < V;
            bad |= !here && idx[b] != -1;
            col[b] = here ? static_cast<int32_t>(idx[b]) : -1;
        }
    }
    bad = G::any(bad);  // (and the barrier is initialised)
    if (G::any(!mbar_wait(&copy_bar[group], 0))) {
        report(p.dev_status, GBCE_DEV_TIMEOUT);
        mbar_wait(&copy_bar[group], 0);
        wait_for_count();
        return;
    }
    if (kList && bad) {
        if (tid == 0)
            report(p.dev_status, GBCE_DEV_BAD_INDEX);
        state = kRowInvalid;
        fill();
        return;
    }

    // the listed logits, and -inf in their place
    const float inf = __builtin_huge_valf();
    bool nan_t = kList && !(rest < inf), nan_x = false;
    LedSum teacher = {kNegInf, 0.0f}, student = {kNegInf, 0.0f};
    const auto exp_t = [](float d) { return expf(d); };
    const auto exp_c = [&](float d) { return ex2(scaled(d, c)); };
    float xy = 0.0f;
    if constexpr (kList) {
#pragma unroll
        for (int b = 0; b < KE && b * NT < K; ++b)
            x[b] = col[b] >= 0 ? as_float(buf[phase + col[b]]) : kNegInf;
        G::sync();
        // an index listed twice: of the entries that leave their numbers at a
        // column only one finds its own there
#pragma unroll
        for (int b = 0; b < KE && b * NT < K; ++b)
            if (col[b] >= 0)
                buf[phase + col[b]] = tag_as(T(), tid + b * NT);
        G::sync();
        bool twice = false;
#pragma unroll
        for (int b = 0; b < KE && b * NT < K; ++b)
            if (col[b] >= 0)
                twice |= tag_of(buf[phase + col[b]]) != tid + b * NT;
        twice = G::any(twice);
#pragma unroll
        for (int b = 0; b < KE && b * NT < K; ++b) {
            if (col[b] >= 0)
                buf[phase + col[b]] = neg_inf_as(T());
            nan_t |= col[b] >= 0 && !(tau[b] < inf);
            tau[b] = col[b] >= 0 ? (twice ? tau[b] : teacher_logit(tau[b], inv_t)) : kNegInf;
        }
        if (twice) {
            // the first of several takes their sum, in entry order; the others go
#pragma unroll
            for (int b = 0; b < KE; ++b)
                if (tid + b * NT < K) {
                    list_col[tid + b * NT] = col[b];
                    list_tau[tid + b * NT] = tau[b];
                }
            G::sync();
            float highest = kNegInf;
            for (int j = 0; j < K; ++j)
                highest = fmaxf(highest, list_tau[j]);
            rest = rest_logit(rest, highest, inv_t);
            G::sync();
#pragma unroll
            for (int b = 0; b < KE; ++b)
                if (tid + b * NT < K) {
                    tau[b] = teacher_logit(tau[b], highest, inv_t);
                    list_tau[tid + b * NT] = tau[b];
                }
            G::sync();
#pragma unroll 1
            for (int b = 0; b < KE && b * NT < K; ++b) {
                const int k = tid + b * NT;
                if (k >= K || list_col[k] < 0)
                    continue;
                const int32_t own = list_col[k];
                float top = kNegInf, sum = 0.0f;
                bool first = true, more = false;
                for (int j = 0; j < K; ++j)
                    if (j != k && list_col[j] == own)
                        (j < k ? first : more) = j > k;  // (an earlier one: not the first)
                if (first && more) {
                    for (int j = k; j < K; ++j)
                        if (list_col[j] == own)
                            top = fmaxf(top, list_tau[j]);
                    for (int j = k; j < K; ++j)
                        if (list_col[j] == own && list_tau[j] != kNegInf)
                            sum += expf(list_tau[j] - top);
                }
#pragma unroll
                for (int i = 0; i < KE; ++i)
                    if (i == b) {
                        col[i] = first ? col[i] : -1;
                        if (first && more)
                            tau[i] = sum > 0.0f ? top + logf(sum) : kNegInf;
                    }
            }
        }
#pragma unroll
        for (int b = 0; b < KE && b * NT < K; ++b)
            if (col[b] >= 0) {
                nan_x |= x[b] != x[b] || x[b] == inf;
                teacher.merge(tau[b], 0.0f, exp_t);
                student.merge(x[b], 0.0f, exp_c);
            }
        if (tid == 0)
            teacher.merge(rest, 0.0f, exp_t);
    } else {
        xy = as_float(buf[phase + y]);
        G::sync();
        if (tid == 0)
            buf[phase + y] = neg_inf_as(T());
    }
    G::sync();

    // the rest's sum, and everybody's part of the lists'
    const uint4 *vec = reinterpret_cast<const uint4 *>(buf);
    if (kStats) {
        constexpr int U = 4;
        RestStats st;
        const uint4 none = all_neg_inf(T());
        for (int v = tid; v < nv; v += U * NT) {
            uint4 raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                raw[u] = v + u * NT < nv ? vec[v + u * NT] : none;
#pragma unroll
            for (int u = 0; u < U; u += 2)
                rest_take<T>(st, raw[u], raw[u + 1], FastVec<T>::vmax(raw[u], raw[u + 1]), c, p.far);
        }
        m = st.m;
        s = st.sum();
        if (s != s)  // (a thread that met only NaN has no max: its NaN must still count)
            m = fmaxf(m, 0.0f);
        warp_merge_rest(m, s, c, st.residual(c));
    }
    int nans = 0;
    const bool listing = kList && warp * 32 < K;  // the warp has entries (the first one the rest too)
    if (listing) {
        teacher.warp_merge(exp_t);
        student.warp_merge(exp_c);
        nans = (__any_sync(0xffffffffu, nan_t) ? 1 : 0) | (__any_sync(0xffffffffu, nan_x) ? 2 : 0);
    }
    if (W > 1 && (kStats || kList)) {
        if (lane == 0)
            partial[warp] = {m, s, teacher.m, teacher.s, student.m, student.s, nans};
        __syncthreads();
        const ShortPartial in =
            lane < W ? partial[lane]
                     : ShortPartial{kNegInf, 0.0f, kNegInf, 0.0f, kNegInf, 0.0f, 0};
        if (kStats) {
            m = in.m;
            s = in.s;
            warp_merge_rest(m, s, c);
        }
        if (kList) {
            teacher = {in.teacher_m, in.teacher_s};
            student = {in.student_m, in.student_s};
            teacher.warp_merge(exp_t);
            student.warp_merge(exp_c);
            nans = __reduce_or_sync(0xffffffffu, in.nans);
        }
    }
    if (kList && ((nans & 1) != 0 || teacher.m == kNegInf)) {
        state = (nans & 1) != 0 ? kRowInvalid : kRowSkip;
        fill();
        return;
    }
    if (nans & 2) {  // a NaN (or +inf) among the listed logits: the row has no softmax
        student.m = 0.0f;
        student.s = kQuietNan;
    }
    if (kStats && p.rest_state_out != nullptr && tid == 0) {
        p.rest_state_out[2 * r] = m;
        p.rest_state_out[2 * r + 1] = s;
    }

    // The kernel after this one (the losses' sum, the pairs) may take its place; it
    // waits for this one's outputs.
    launch_dependents();
    wait_for_count();
    if (kGrad && p.n_items != nullptr && p.reduction == GBCE_MEAN)
        n_items = *p.n_items;

    // the loss of a token, and what the sweep over the unlisted columns is scaled by
    const float gt = kGrad ? scaled(post_upstream(p, r, n_items), inv_t) : 0.0f;
    const float lt = kList ? log1pf(teacher.s) : 0.0f;
    const float lp_rest = rest == kNegInf ? kNegInf : (rest - teacher.m) - lt;
    float gs = 0.0f, dy = 0.0f;
    if (kList) {
        if (kGrad)
            gs = gt * rest_gap(m, s, student.m, student.s, lp_rest, c, inv_t);
    } else {
        const TokenTerms q = token_terms(m, s, xy, inv_t);
        float slope = gt;
        if (kStats && p.logp_out != nullptr && tid == 0)
            p.logp_out[r] = q.lp;
        if (OP == kOpPolicy) {
            float loss, dlp;
            policy_row(p.policy, adv, old_lp, ref_lp, q.lp, loss, dlp);
            if (tid == 0)
                p.loss_rows[r] = loss;
            slope *= dlp;
        }
        dy = slope * q.other;
        gs = -dy;
    }

    if (kGrad) {
        const GradConsts gk = rest_consts<T>(m, s, c.hi + c.lo, gs);
        const RowGeom gd = row_geom<T>(drow, V);
        const int first = phase + static_cast<int>(gd.head), sh = first & (VEC - 1);
        const uint4 *from = vec + first / VEC;
        uint4 *body = reinterpret_cast<uint4 *>(drow + gd.head);
        const int n = static_cast<int>(gd.nvec);
        if (tid < gd.head)
            E::store(drow + tid, grad_scalar(as_float(buf[phase + tid]), gk));
        if (gd.tail0 + tid < V)
            E::store(drow + gd.tail0 + tid, grad_scalar(as_float(buf[phase + gd.tail0 + tid]), gk));
        constexpr int32_t kNoLabel = 0x7fffffff;
        if (sh == 0) {
#pragma unroll 4
            for (int v = tid; v < n; v += NT)
                st_cs_v4(body + v, GradVec<T>::run(from[v], kNoLabel, gk));
        } else {
            // (the last vector ends inside the row, so its second half is in the buffer)
#pragma unroll 2
            for (int v = tid; v < n; v += NT)
                st_cs_v4(body + v,
                         GradVec<T>::run(shifted<T>(from[v], from[v + 1], sh), kNoLabel, gk));
        }
        G::sync();  // the listed columns, over what the sweep stored there
        if (!kList && tid == 0)
            E::store(drow + y, dy);
    }
    if constexpr (kList) {
        float kl = 0.0f;
        if (listing) {
            const StudentRow q = student_row(m, s, student.m, student.s, c, inv_t);
            if (tid == 0)
                kl = entry_terms(lp_rest, q.log_rest).kl;
#pragma unroll
            for (int b = 0; b < KE && b * NT < K; ++b) {
                if (col[b] < 0)
                    continue;
                const EntryTerms t =
                    entry_terms((tau[b] - teacher.m) - lt, student_logp(q, x[b], inv_t));
                kl += t.kl;
                if (kGrad)
                    E::store(drow + col[b], gt * t.gap);
            }
            kl = warp_sum(kl);
        }
        if (!kStats)
            return;
        if (W > 1 && K > 32) {
            if (lane == 0)
                partial_kl[warp] = kl;
            G::sync();
            kl = warp_sum(lane < W ? partial_kl[lane] : 0.0f);
        }
        if (tid == 0)
            p.loss_rows[r] = kl;
    }
}

// Rows of a batch up to which no kernel is launched to count the kept ones: where
// every CTA needs the number (a mean's gradient; us, counted by every CTA / before:
// policy loss, 1000 x 2000 7.7 / 7.5 and one launch less for the host, 2000 x 14000 30 / 25),
// and where only the call's result does, for which one CTA counts.
constexpr int64_t kShortSelfCount = 1024, kShortOneCount = 16384;

template <typename T, int OP, int PASS, int W>
cudaError_t launch_short_as(PostParams p, cudaStream_t stream)
{
    static std::atomic<uint64_t> attr_done{0};
    auto kernel = post_short_kernel<T, OP, PASS, W>;
    const int smem = short_smem<T, W>(p.vocab, OP, p.k);
    cudaError_t err = ensure_smem_attr(kernel, kShortSmemMax, attr_done);
    if (err != cudaSuccess)
        return err;
    int ordered = 0;
    const bool each = PASS != kPassFwd && p.reduction == GBCE_MEAN;
    if (p.n_items_out != nullptr && p.rows > (each ? kShortSelfCount : kShortOneCount)) {
        err = OP == kOpDistill
                  ? launch_count_mask(p.row_mask, p.rows, p.n_items_out, nullptr, stream)
                  : launch_count_items(p.labels, p.rows, p.ignore_index, p.n_items_out, nullptr,
                                       nullptr, nullptr, stream);
        if (err != cudaSuccess)
            return err;
        p.n_items = p.n_items_out;
        p.n_items_out = nullptr;
        ordered = 1;
    }
    using G = RowGroup<W>;
    const PostLaunch l((p.rows + G::kRows - 1) / G::kRows, G::kCta, smem, 1, stream);
    err = cudaLaunchKernelEx(&l.cfg, kernel, static_cast<const PostParams>(p), ordered);
    note_launches(1);
    return err != cudaSuccess ? err : cudaGetLastError();
}

// How many warps a row gets.  One warp each keeps most rows in flight where there
// are more of them than one wave of CTAs.
template <typename T, int OP, int PASS>
cudaError_t launch_short_pass(const PostParams &p, cudaStream_t stream)
{
    const int64_t row = p.vocab * static_cast<int64_t>(sizeof(T));
    if (row <= kShortWarpBytes && p.rows > kShortFewRows)
        return launch_short_as<T, OP, PASS, 1>(p, stream);
    if (row <= kShortMidBytes)
        return launch_short_as<T, OP, PASS, 4>(p, stream);
    return launch_short_as<T, OP, PASS, 8>(p, stream);
}

template <typename T>
cudaError_t launch_post_short(const PostParams &p, int op, int pass, cudaStream_t stream)
{
    if (op == kOpPolicy)
        return launch_short_pass<T, kOpPolicy, kPassFused>(p, stream);
    if (op == kOpToken)
        return pass == kPassFwd ? launch_short_pass<T, kOpToken, kPassFwd>(p, stream)
                                : launch_short_pass<T, kOpToken, kPassBwd>(p, stream);
    if (pass == kPassFwd)
        return launch_short_pass<T, kOpDistill, kPassFwd>(p, stream);
    if (pass == kPassBwd)
        return launch_short_pass<T, kOpDistill, kPassBwd>(p, stream);
    return launch_short_pass<T, kOpDistill, kPassFused>(p, stream);
}

}  // namespace gbce
