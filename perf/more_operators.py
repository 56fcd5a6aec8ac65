"""The post-training losses over [rows, vocab] logits, case by case.

Three operators, each with its gradient with respect to the logits:

* distillation from a teacher's top logits (``distill_fwd``, ``distill_bwd``,
  ``distill_fwd_bwd_fused``): KL of the teacher's distribution over its listed
  tokens, and a bucket for its other tokens where their mass is given;
* the clipped policy loss with a KL term (``policy_loss_fwd_bwd_fused``, and
  ``policy_loss`` from log-probs);
* the preference loss of paired sequences (``preference_loss_fwd_bwd_fused``,
  and ``preference_loss`` from log-probs).

Each case is run in a plain form (elementary torch operations in fp32, sums
over a sequence in fp64, rounded once) or, with ``own`` set, through the
package's entry points; ``exact`` gives the same outputs from the definitions
in fp64.
"""

import math

import torch

own = False  # set by whoever loads this file

IGNORE = -100
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # ----------------------------------------- distillation from a teacher's top logits
        # a unit-test sized fp32 student with sixteen teacher tokens a row: all latency
        dict(name="distill_small_fp32", op="distill", rows=64, vocab=4096, k=16, dtype="fp32",
             masked=0.1, rest=False, ragged=False, temperature=1.0, reduction="mean"),
        # a decoding batch of students trained on-policy: few rows of the benchmark's vocabulary
        dict(name="distill_few_rows", op="distill", rows=48, vocab=152064, k=20, dtype="bf16",
             masked=0.0, rest=True, ragged=True, temperature=1.0, reduction="none"),
        # odd everything: rows of a wider buffer, nucleus-truncated lists of up to 50, T = 2
        dict(name="distill_odd_strided", op="distill", rows=613, vocab=40001, k=50, dtype="bf16",
             masked=0.1, rest=True, ragged=True, temperature=2.0, reduction="sum", pad=7),
        # an autograd step: the forward, then the backward with the loss's own upstream gradient
        dict(name="distill_step_fp32", op="distill_step", rows=512, vocab=32768, k=100, dtype="fp32",
             masked=0.15, rest=True, ragged=False, temperature=0.7, reduction="mean"),
        # the packed training step: 8 sequences of 1024 tokens, the teacher's 64 top tokens
        dict(name="distill_packed", op="distill", rows=8192, vocab=152064, k=64, dtype="bf16",
             masked=0.05, rest=False, ragged=False, temperature=1.0, reduction="mean"),
        # ----------------------------------------- the clipped policy loss with a KL term
        # a unit-test sized fp32 policy: all latency
        dict(name="policy_small_fp32", op="policy", rows=64, vocab=4096, dtype="fp32", ignored=0.1,
             clip_low=0.2, clip_high=0.2, beta=0.04, temperature=1.0, reduction="mean"),
        # completions cropped to 1922 rows of which about a third are the policy's own tokens
        dict(name="policy_sparse", op="policy", rows=1922, vocab=32768, dtype="bf16", ignored=0.66,
             clip_low=0.2, clip_high=0.28, beta=0.0, temperature=0.9, reduction="sum", pad=5),
        # the packed policy step, old and reference log-probs at hand
        dict(name="policy_packed", op="policy", rows=8192, vocab=152064, dtype="bf16", ignored=0.15,
             clip_low=0.2, clip_high=0.2, beta=0.04, temperature=0.9, reduction="mean"),
        # the same loss where the log-probs are at hand already (a linear or vocabulary-parallel
        # head made them): a long rollout buffer
        dict(name="policy_from_logp", op="policy_logp", rows=65536, vocab=1, dtype="fp32", ignored=0.3,
             clip_low=0.2, clip_high=0.28, beta=0.01, temperature=1.0, reduction="mean"),
        # ----------------------------------------- the preference loss of paired sequences
        # two pairs of short answers, fp32: all latency
        dict(name="preference_small_fp32", op="preference", rows=64, vocab=4096, pairs=2,
             dtype="fp32", ignored=0.2, beta=0.1, margin=0.0, smoothing=0.0, kind="sigmoid",
             average=False, reference=True, temperature=1.0, reduction="mean"),
        # ragged answers (empty ones among them) of an odd vocabulary, length-normalised, no reference
        dict(name="preference_odd", op="preference", rows=701, vocab=50257, pairs=9, dtype="bf16",
             ignored=0.3, beta=2.0, margin=0.25, smoothing=0.1, kind="sigmoid", average=True,
             reference=False, temperature=1.0, reduction="sum", pad=3),
        # a packed batch of four pairs, about 512 tokens an answer
        dict(name="preference_packed", op="preference", rows=4096, vocab=152064, pairs=4,
             dtype="bf16", ignored=0.25, beta=0.1, margin=0.0, smoothing=0.0, kind="sigmoid",
             average=False, reference=True, temperature=1.0, reduction="mean"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["distill", "distill", "distill_step", "policy", "policy", "policy_logp",
                     "preference", "preference"])
    dtype = "fp32" if op == "policy_logp" or rng.random() < 0.35 else "bf16"
    rows = _spread(rng, 1, 2048 if dtype == "fp32" else 8192)
    vocab = _spread(rng, 64, 152064)
    case = dict(op=op, rows=rows, vocab=vocab, dtype=dtype,
                temperature=rng.choice([1.0, 0.9, 0.7, 1.3, 2.0]),
                reduction=rng.choice(["mean", "sum", "none"]), pad=rng.choice([0, 0, 5, 8]))
    if op in ("distill", "distill_step"):
        case.update(k=min(_spread(rng, 1, 256), vocab // 2), masked=rng.choice([0.0, 0.15, 0.6]),
                    rest=rng.random() < 0.5, ragged=rng.random() < 0.5)
    if op in ("policy", "policy_logp"):
        case.update(ignored=rng.choice([0.0, 0.15, 0.7]), beta=rng.choice([0.0, 0.01, 0.2]),
                    clip_low=rng.choice([0.1, 0.2]), clip_high=rng.choice([0.2, 0.28]))
    if op == "policy_logp":
        case.update(rows=_spread(rng, 1, 262144), vocab=1, temperature=1.0, pad=0)
    if op == "preference":
        case["rows"] = rows = min(rows, 4096)
        case.update(pairs=min(_spread(rng, 1, 64), max(1, rows // 2)), ignored=rng.choice([0.0, 0.3, 0.6]),
                    beta=rng.choice([0.05, 0.1, 2.0]), margin=rng.choice([0.0, 0.5]),
                    smoothing=rng.choice([0.0, 0.1]), kind=rng.choice(["sigmoid", "sigmoid", "squared"]),
                    reference=rng.random() < 0.7)
        # a sum of log-probs under a steep loss has no upstream gradient left to measure
        case["average"] = case["beta"] > 1.0 or case["kind"] == "squared" or rng.random() < 0.3
    return case


# --------------------------------------------------------------------- inputs

def _rand(g, *shape):
    return torch.rand(shape, generator=g, device="cuda")


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _logits(case, g):
    """Logits of std 2.2, rows of a buffer `pad` columns wider."""
    rows, vocab, pad = case["rows"], case["vocab"], int(case.get("pad", 0))
    x = torch.empty((rows, vocab + pad), dtype=DTYPES[case["dtype"]], device="cuda")
    for part in x.split(1024):
        part.copy_(_randn(g, *part.shape).mul_(2.2))
    return x[:, :vocab]


def _lead(rows, g):
    """How far a row's chosen token leads: most by a few nats, one row in twenty by 8 to 12, one in
    twenty past fp32's 1 - p (17 to 50)."""
    u, w = _rand(g, rows), _rand(g, rows)
    return torch.where(u < 0.05, 8.0 + 4.0 * w, torch.where(u > 0.95, 17.0 + 33.0 * w, 9.0 * w))


def _left_out(rows, share, g):
    """Which rows are left out; the first never is."""
    skip = _rand(g, rows) < share
    skip[0] = False
    return skip


def _labels(case, x, g):
    """The tokens that were sampled, a few nats ahead of the noise; IGNORE at the prompts' rows."""
    rows, T = case["rows"], case["temperature"]
    tok = (_rand(g, rows).double() * case["vocab"]).long().clamp_(max=case["vocab"] - 1)
    lead = (_lead(rows, g) * T + 2.2 * 2.0).unsqueeze(1)
    x.scatter_(1, tok.unsqueeze(1), lead.to(x.dtype))
    return tok.masked_fill(_left_out(rows, case["ignored"], g), IGNORE)


def _recorded_logp(case, x, labels):
    """log-probs of the labels as a recording of them would hold (fp32)."""
    out = torch.zeros(case["rows"], device="cuda")
    for lo in range(0, case["rows"], 1024):
        z = x[lo:lo + 1024].float() / case["temperature"]
        lab = labels[lo:lo + 1024].clamp(min=0).unsqueeze(1)
        out[lo:lo + 1024] = z.gather(1, lab).squeeze(1) - torch.logsumexp(z, 1)
    return out


def _teacher(case, x, g):
    """The teacher's top tokens (spread over the vocabulary, most likely first), its logits there,
    and the student's logits moved to about the same values."""
    rows, V, K, T = case["rows"], case["vocab"], case["k"], case["temperature"]
    slots = torch.arange(K, device="cuda").double()
    col = ((slots + _rand(g, rows, K).double()) * (V / K)).floor().long()
    lo = (slots * (V / K)).ceil().long()
    col = torch.minimum(torch.maximum(col, lo), torch.cat([lo[1:] - 1, lo.new_tensor([V - 1])]))
    order = torch.argsort(_rand(g, rows, K), 1)
    index = col.gather(1, order)
    t = 9.0 - 1.5 * torch.log1p(slots).float() + 0.3 * _randn(g, rows, K)
    t[:, 0] += _lead(rows, g)
    t = t.sort(1, descending=True).values * T
    x.scatter_(1, index, (t + 0.7 * T * _randn(g, rows, K)).to(x.dtype))
    if case["ragged"]:
        keep = (_rand(g, rows) * K).ceil().long().clamp_(min=1)
        gone = torch.arange(K, device="cuda") >= keep.unsqueeze(1)
        index = index.masked_fill(gone, -1)
        t = t.masked_fill(gone, math.nan)   # whatever a buffer holds behind a list's end
    rest = None
    if case["rest"]:
        kept = torch.logsumexp((t / T).masked_fill(index < 0, -math.inf), 1)
        rest = kept - 0.5 - 6.0 * _rand(g, rows)
    return index, t, rest


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    rows, op, T = case["rows"], case["op"], case["temperature"]
    st = dict(op=op, temperature=T, reduction=case["reduction"])
    if op == "policy_logp":
        live = ~_left_out(rows, case["ignored"], g)
        st["mask"] = live.to(torch.uint8)
        logp = -_rand(g, rows).mul_(6.0).pow_(2).mul_(0.3)
    else:
        st["logits"] = _logits(case, g)
    if op in ("distill", "distill_step"):
        st["index"], st["teacher"], st["rest"] = _teacher(case, st["logits"], g)
        skip = _left_out(rows, case["masked"], g)
        st["mask"] = (~skip).to(torch.uint8)
        n = rows
    elif op in ("policy", "preference"):
        st["labels"] = _labels(case, st["logits"], g)
        logp = _recorded_logp(case, st["logits"], st["labels"])
        n = rows
    if op in ("policy", "policy_logp"):
        lo, hi = case["clip_low"], case["clip_high"]
        # the policy moved by a few percent since the tokens were sampled, past the clip for some;
        # none sits within 1e-3 of a clip's border, where rounding alone would choose the side
        d = 0.15 * _randn(g, rows)
        for edge in (math.log1p(-lo), math.log1p(hi)):
            d = torch.where((d - edge).abs() < 1e-3, torch.full_like(d, edge + 2e-3), d)
        # (in fp64: a recorded log-prob near 0 holds the move only there)
        st["old_logp"] = (logp.double() - d.double()).float()
        st["ref_logp"] = logp + 0.2 * _randn(g, rows) if case["beta"] else None
        st["advantages"] = _randn(g, rows)
        st.update(clip_low=lo, clip_high=hi, beta=case["beta"])
        if op == "policy_logp":
            st["logp"] = logp
        n = rows
    if op == "preference":
        pairs = case["pairs"]
        cuts = (_rand(g, 2 * pairs - 1).double() * (rows + 1)).long().sort().values
        if pairs > 4:
            cuts[1] = cuts[0]      # an answer of no tokens
        # a few rows behind the last answer belong to none (a padded batch)
        end = torch.tensor([rows - min(3, rows // 8)], device="cuda")
        st["offsets"] = torch.cat([end.new_zeros(1), cuts, end]).clamp_(max=int(end))
        st["pairs"] = pairs
        # the reference policy's log-probs of the same tokens
        st["ref_logp"] = logp + 0.2 * _randn(g, rows) if case["reference"] else None
        for name in ("beta", "margin", "smoothing", "kind", "average"):
            st[name] = case[name]
        n = pairs
    st["grad_out"] = {"none": (0.5 + _rand(g, n)) / n, "sum": torch.full((1,), 1.0 / n, device="cuda"),
                      "mean": torch.ones(1, device="cuda")}[case["reduction"]]
    return st


# ----------------------------------------------------------------- plain forms

def _softplus(a):
    return a.clamp(min=0) + torch.log1p(torch.exp(-a.abs()))


def _logsumexp(x, dim):
    m = x.amax(dim, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    return torch.log(torch.exp(x - m).sum(dim)) + m.squeeze(dim)


def _reduce(per, n, reduction):
    return {"none": per, "sum": per.sum(dtype=torch.float64).to(per.dtype),
            "mean": (per.sum(dtype=torch.float64) / n).to(per.dtype)}[reduction]


def _upstream(st, live, n):
    return st["grad_out"] / (n if st["reduction"] == "mean" else 1) * live


def _by_sequence(v, live, offsets):
    """Sums of v and counts of live over each sequence's rows."""
    zero = v.new_zeros(1)
    total = torch.cat([zero, torch.cumsum(v, 0)])
    count = torch.cat([zero, torch.cumsum(live.to(v.dtype), 0)])
    lo, hi = offsets[:-1], offsets[1:]
    return total[hi] - total[lo], count[hi] - count[lo]


def _plain_distill(st):
    T, idx = st["temperature"], st["index"]
    live, here = st["mask"].bool(), st["index"] >= 0
    col = torch.where(here, idx, idx[:, :1])
    z = st["logits"].float() / T
    zl = z.gather(1, col).masked_fill(~here, -math.inf)
    z_rest = _logsumexp(z.scatter(1, col, -math.inf), 1)
    lse = torch.logaddexp(z_rest, _logsumexp(zl, 1))
    t = (st["teacher"] / T).masked_fill(~here, -math.inf)
    rest = st["rest"] if st["rest"] is not None else torch.full_like(lse, -math.inf)
    t_lse = torch.logaddexp(_logsumexp(t, 1), rest)
    logp = torch.cat([t, rest.unsqueeze(1)], 1) - t_lse.unsqueeze(1)
    logq = torch.cat([zl, z_rest.unsqueeze(1)], 1) - lse.unsqueeze(1)
    p = torch.exp(logp)
    kl = torch.where(p > 0, p * (logp - logq), torch.zeros_like(p)).sum(1)
    n = live.sum()
    loss = _reduce(torch.where(live, kl, torch.zeros_like(kl)), n, st["reduction"])
    scale = -torch.expm1(logp[:, -1] - logq[:, -1])
    dz = torch.exp(z.sub_(lse.unsqueeze(1))).mul_(scale.unsqueeze(1))
    dl = (torch.exp(logq) - p)[:, :-1]
    dz.scatter_(1, col, torch.where(here, dl, dl[:, :1]))
    dz *= (_upstream(st, live, n) / T).unsqueeze(1)
    dz[~live] = 0.0
    return dict(loss=loss, dlogits=dz.to(st["logits"].dtype), n_items=n)


def _plain_logp(st):
    """logits / T, their logsumexp and the log-probs of the labels, taken from the other columns."""
    live = st["labels"] != IGNORE
    lab = st["labels"].masked_fill(~live, 0).unsqueeze(1)
    z = st["logits"].float() / st["temperature"]
    zy = z.gather(1, lab)
    others = _logsumexp(z.scatter(1, lab, -math.inf), 1)
    logp = -_softplus(others - zy[:, 0])
    return z, lab, live, torch.where(live, logp, torch.zeros_like(logp)), torch.logaddexp(others, zy[:, 0])


def _plain_policy_terms(st, logp, live):
    """Each row's loss and its derivative with respect to log p."""
    A, beta = st["advantages"], st["beta"]
    ratio = torch.exp(logp - st["old_logp"])
    clipped = ratio.clamp(1.0 - st["clip_low"], 1.0 + st["clip_high"])
    per = -torch.minimum(ratio * A, clipped * A)
    d = torch.where(ratio * A <= clipped * A, -A * ratio, torch.zeros_like(A))
    if beta:
        away = st["ref_logp"] - logp
        per = per + beta * (torch.expm1(away) - away)
        d = d - beta * torch.expm1(away)
    zero = torch.zeros_like(per)
    return torch.where(live, per, zero), torch.where(live, d, zero)


def _plain_preference_terms(st, logp, live):
    """Pair losses, sequence scores, and the derivative of each pair's loss by its rows' log-probs."""
    off, beta = st["offsets"], st["beta"]
    pairs = st["pairs"]
    r = torch.arange(logp.numel(), device=logp.device)
    seq = torch.searchsorted(off, r, right=True) - 1
    inside = (seq < 2 * pairs) & live
    seq = seq.clamp(max=2 * pairs - 1)
    ratio = logp.double() - (st["ref_logp"].double() if st["ref_logp"] is not None else 0.0)
    score, count = _by_sequence(torch.where(inside, ratio, torch.zeros_like(ratio)), inside, off)
    weight = 1.0 / count.clamp(min=1) if st["average"] else torch.ones_like(count)
    score = score * weight
    h = score[:pairs] - score[pairs:]
    if st["kind"] == "squared":
        e = h - 1.0 / (2.0 * beta)
        per, dh = e * e, 2.0 * e
    else:
        h = beta * (h - st["margin"])
        s = st["smoothing"]
        per = (1.0 - s) * _softplus(-h) + s * _softplus(h)
        dh = beta * (s / (1.0 + torch.exp(-h)) - (1.0 - s) / (1.0 + torch.exp(h)))
    d = torch.cat([dh, -dh]) * weight
    up = st["grad_out"].double() / (pairs if st["reduction"] == "mean" else 1)
    up = up.expand(pairs) if up.numel() == 1 else up
    drow = (d * torch.cat([up, up]))[seq] * inside
    return per.float(), score.float(), drow.float(), inside


def _plain(st):
    op, T = st["op"], st["temperature"]
    if op in ("distill", "distill_step"):
        return _plain_distill(st)
    if op == "policy_logp":
        live = st["mask"].bool()
        per, d = _plain_policy_terms(st, st["logp"], live)
        n = live.sum()
        return dict(loss=_reduce(per, n, st["reduction"]), dlogp=d * _upstream(st, live, n), n_items=n)
    z, lab, live, logp, lse = _plain_logp(st)
    if op == "policy":
        per, d = _plain_policy_terms(st, logp, live)
        n = live.sum()
        out = dict(loss=_reduce(per, n, st["reduction"]), logp=logp, n_items=n)
        d = d * _upstream(st, live, n)
    else:
        per, score, d, live = _plain_preference_terms(st, logp, live)
        logp = torch.where(live, logp, torch.zeros_like(logp))
        out = dict(loss=_reduce(per, per.numel(), st["reduction"]), logp=logp, seq_score=score)
    dz = torch.exp(z.sub_(lse.unsqueeze(1))).scatter_(1, lab, torch.expm1(logp).unsqueeze(1))
    dz *= (-d / T).unsqueeze(1)
    dz[~live] = 0.0
    return dict(out, dlogits=dz.to(st["logits"].dtype))


def run(st):
    if not own:
        return _plain(st)
    import cross_entropy_gb300 as gbce

    op, T, red = st["op"], st["temperature"], st["reduction"]
    if op == "distill":
        r = gbce.distill_fwd_bwd_fused(st["logits"], st["index"], st["teacher"], st["rest"],
                                       st["grad_out"], T, st["mask"], red)
        return dict(loss=r.loss, dlogits=r.dlogits, n_items=r.n_items)
    if op == "distill_step":
        f = gbce.distill_fwd(st["logits"], st["index"], st["teacher"], st["rest"], T, st["mask"], red)
        d = gbce.distill_bwd(st["logits"], st["index"], st["teacher"], st["rest"], st["grad_out"],
                             f.rest_state, f.n_items, T, st["mask"], red)
        return dict(loss=f.loss, dlogits=d, n_items=f.n_items)
    if op == "policy":
        r = gbce.policy_loss_fwd_bwd_fused(st["logits"], st["labels"], st["advantages"],
                                           st["old_logp"], st["ref_logp"], st["grad_out"],
                                           clip_low=st["clip_low"], clip_high=st["clip_high"],
                                           kl_beta=st["beta"], temperature=T, reduction=red)
        return dict(loss=r.loss, logp=r.logp, n_items=r.n_items, dlogits=r.dlogits)
    if op == "policy_logp":
        r = gbce.policy_loss(st["logp"], st["advantages"], st["old_logp"], st["ref_logp"],
                             st["grad_out"], st["mask"], clip_low=st["clip_low"],
                             clip_high=st["clip_high"], kl_beta=st["beta"], reduction=red)
        return dict(loss=r.loss, dlogp=r.dlogp, n_items=r.n_items)
    r = gbce.preference_loss_fwd_bwd_fused(st["logits"], st["labels"], st["offsets"], st["ref_logp"],
                                           st["grad_out"], beta=st["beta"], margin=st["margin"],
                                           label_smoothing=st["smoothing"], kind=st["kind"],
                                           average=st["average"], temperature=T, reduction=red)
    return dict(loss=r.loss, logp=r.logp, seq_score=r.seq_score, dlogits=r.dlogits)


# ------------------------------------------------------------------ what it costs

def work(case):
    rows, V, op = case["rows"], case["vocab"], case["op"]
    e = 2 if case["dtype"] == "bf16" else 4
    live = max(1.0, rows * (1.0 - case.get("ignored", case.get("masked", 0.0))))
    if op == "policy_logp":
        return dict(bytes=rows * (5.0 + 16.0 + (4.0 if case["beta"] else 0.0)), flops=rows * 20.0)
    # the logits read once, their gradient written once (zeros for the rows left out)
    side = live * case["k"] * 12.0 if op in ("distill", "distill_step") else rows * 24.0
    return dict(bytes=(live + rows) * V * e + side, flops=live * V * 8.0)


# ---------------------------------------------------------------- 64 bits

def _exact_rows(x, T, col):
    """For rows x: q of every column, and of the listed columns col [rows, K] (K may differ by row:
    entries repeat the first) log q, with their complement's sum taken over the other columns."""
    z = x.double() / T
    top = z.max(1, keepdim=True).values
    e = torch.exp(z - top)
    q = e / e.sum(1, keepdim=True)
    rest = e.scatter(1, col, 0.0).sum(1)
    return z, top.squeeze(1), e, q, rest


def _exact_distill(case, st):
    T, rows, red = case["temperature"], case["rows"], case["reduction"]
    live = torch.nonzero(st["mask"]).squeeze(1)
    n = live.numel()
    per = torch.zeros(rows, dtype=torch.float64, device="cuda")
    dx = torch.zeros((rows, case["vocab"]), dtype=torch.float64, device="cuda")
    up = st["grad_out"].double().expand(rows) / (n if red == "mean" else 1)
    for r in live.split(256):
        idx = st["index"][r]
        here = idx >= 0
        col = torch.where(here, idx, idx[:, :1])
        z, top, e, q, rest = _exact_rows(st["logits"][r], T, col)
        total = e.sum(1)
        # the teacher's weights, the bucket of its other tokens last
        w = torch.where(here, st["teacher"][r].double() / T, torch.full_like(top[:, None], -math.inf))
        if st["rest"] is not None:
            w = torch.cat([w, st["rest"][r].double().unsqueeze(1)], 1)
        else:
            w = torch.cat([w, torch.full_like(top[:, None], -math.inf)], 1)
        p = torch.softmax(w, 1)
        logp = torch.log_softmax(w, 1)
        qb = torch.cat([torch.where(here, q.gather(1, col), torch.zeros_like(p[:, :-1])),
                        (rest / total).unsqueeze(1)], 1)
        logq = torch.cat([z.gather(1, col) - top[:, None] - torch.log(total)[:, None],
                          torch.log(rest / total).unsqueeze(1)], 1)
        per[r] = torch.where(p > 0, p * (logp - logq), torch.zeros_like(p)).sum(1)
        dz = q * ((qb[:, -1] - p[:, -1]) / qb[:, -1]).unsqueeze(1)
        dl = (qb - p)[:, :-1]
        dz.scatter_(1, col, torch.where(here, dl, dl[:, :1]))
        dx[r] = dz * (up[r] / T).unsqueeze(1)
    loss = {"none": per, "sum": per.sum(), "mean": per.sum() / max(n, 1)}[red]
    return dict(loss=loss, dlogits=dx, n_items=st["mask"].long().sum())


def _exact_policy_row(st, lp):
    A = st["advantages"].double()
    ratio = torch.exp(lp - st["old_logp"].double())
    low, high = 1.0 - st["clip_low"], 1.0 + st["clip_high"]
    held = torch.where(A >= 0, ratio > high, ratio < low)
    edge = torch.where(A >= 0, torch.full_like(A, high), torch.full_like(A, low))
    per = -A * torch.where(held, edge, ratio)
    d = torch.where(held, torch.zeros_like(A), -A * ratio)
    if st["beta"]:
        gap = st["ref_logp"].double() - lp
        per = per + st["beta"] * (torch.exp(gap) - 1.0 - gap)
        d = d + st["beta"] * (1.0 - torch.exp(gap))
    return per, d


def _exact_preference_rows(case, st, lp, live):
    off = st["offsets"].tolist()
    pairs = case["pairs"]
    score = torch.zeros(2 * pairs, dtype=torch.float64, device="cuda")
    lift = lp - st["ref_logp"].double() if st["ref_logp"] is not None else lp
    weight = torch.zeros(case["rows"], dtype=torch.float64, device="cuda")
    seq = torch.full((case["rows"],), -1, device="cuda")
    for s in range(2 * pairs):
        rows = slice(off[s], off[s + 1])
        kept = live[rows]
        w = 1.0 / max(int(kept.sum()), 1) if st["average"] else 1.0
        score[s] = (lift[rows] * kept).sum() * w
        weight[rows] = kept * w
        seq[rows] = s
    h = score[:pairs] - score[pairs:]
    F = torch.nn.functional
    if st["kind"] == "squared":
        per, dh = (h - 0.5 / st["beta"]).square(), 2.0 * (h - 0.5 / st["beta"])
    else:
        h, s = st["beta"] * (h - st["margin"]), st["smoothing"]
        per = -(1.0 - s) * F.logsigmoid(h) - s * F.logsigmoid(-h)
        dh = st["beta"] * (s * torch.sigmoid(h) - (1.0 - s) * torch.sigmoid(-h))
    up = st["grad_out"].double().expand(pairs) / (pairs if st["reduction"] == "mean" else 1)
    by_seq = torch.cat([dh * up, -dh * up])
    d = torch.where(seq >= 0, by_seq[seq.clamp(min=0)] * weight, torch.zeros_like(weight))
    return per, score, d, seq >= 0


def exact(case, seed):
    st = prepare(case, seed)
    op, rows, T, red = case["op"], case["rows"], case["temperature"], case["reduction"]
    if op in ("distill", "distill_step"):
        return _exact_distill(case, st)
    if op == "policy_logp":
        live = st["mask"].bool()
        per, d = _exact_policy_row(st, st["logp"].double())
        n = int(live.sum())
        per, d = per * live, d * live * st["grad_out"].double() / (n if red == "mean" else 1)
        loss = {"none": per, "sum": per.sum(), "mean": per.sum() / max(n, 1)}[red]
        return dict(loss=loss, dlogp=d, n_items=live.sum())
    live = st["labels"] >= 0
    lab = st["labels"].clamp(min=0).unsqueeze(1)
    lp = torch.zeros(rows, dtype=torch.float64, device="cuda")
    kept = torch.nonzero(live).squeeze(1)
    for r in kept.split(256):
        z, top, e, q, rest = _exact_rows(st["logits"][r], T, lab[r])
        # log p = -log(1 + (the others' sum) / (the label's own term))
        lp[r] = -torch.log1p(rest * torch.exp(top - z.gather(1, lab[r]).squeeze(1)))
    if op == "policy":
        per, d = _exact_policy_row(st, lp)
        n = int(live.sum())
        per, d = per * live, d * live * st["grad_out"].double() / (n if red == "mean" else 1)
        out = dict(loss={"none": per, "sum": per.sum(), "mean": per.sum() / max(n, 1)}[red], logp=lp,
                   n_items=live.sum())
    else:
        per, score, d, inside = _exact_preference_rows(case, st, lp, live)
        lp = lp * inside
        out = dict(loss={"none": per, "sum": per.sum(), "mean": per.mean()}[red], logp=lp, seq_score=score)
    dx = torch.zeros((rows, case["vocab"]), dtype=torch.float64, device="cuda")
    for r in kept.split(256):
        z, top, e, q, rest = _exact_rows(st["logits"][r], T, lab[r])
        q.scatter_(1, lab[r], -(rest / e.sum(1)).unsqueeze(1))    # p_y - 1
        dx[r] = q * (-d[r] / T).unsqueeze(1)
    return dict(out, dlogits=dx)
