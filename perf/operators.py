"""The operators that start from hidden states and the head's table, case by case.

Three operators over a vocabulary table ``weight`` [vocab, dim]:

* token cross-entropy of ``hidden @ weight.T`` with both gradients
  (``linear_ce_fwd_bwd_fused``), the logits never kept;
* log-probs of gathered tokens of ``hidden @ weight.T``
  (``linear_selective_logsoftmax`` and ``_bwd``), for rollouts, single
  decoded tokens and the policy step;
* the lookup of token rows in that table with a scale and its gradient
  (``embedding_lookup`` and ``_bwd``), alone and added to the head's gradient
  of the same table.

Each case is run in a plain form (elementary torch operations in fp32,
rounded once) or, with ``own`` set, through the package's entry points;
``exact`` gives the same outputs from the definitions in fp64.
"""

import math

import torch

own = False  # set by whoever loads this file

IGNORE = -100
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # ------------------------------------------------ loss and both gradients
        # the smallest training call: a unit-test sized fp32 head, all latency
        dict(name="ce_small_fp32", op="ce", rows=64, vocab=4096, dim=256, dtype="fp32", ignored=0.1,
             temperature=1.0, reduction="mean"),
        # supervised fine-tuning with few supervised tokens: two cropped samples, 256 of 1922 rows
        # labelled, each with the weight 1/256
        dict(name="ce_sparse_sft", op="ce", rows=1922, vocab=4096, dim=1024, dtype="bf16",
             ignored=1.0 - 256.0 / 1922.0, temperature=1.0, reduction="none"),
        # odd everything: a vocabulary and a width that are no multiples of anything, rows of a
        # wider buffer, T below 1
        dict(name="ce_odd_strided", op="ce", rows=613, vocab=40001, dim=1001, dtype="bf16",
             ignored=0.1, temperature=0.9, reduction="sum", pad=7),
        # the packed training step: 8 sequences of 1024 tokens, the benchmark's vocabulary
        dict(name="ce_packed", op="ce", rows=8192, vocab=152064, dim=4096, dtype="bf16",
             ignored=0.05, temperature=1.0, reduction="mean"),
        # ------------------------------------------------ log-probs of gathered tokens
        # serving: one decoded token's log-prob, which reads the whole table
        dict(name="logp_one_token", op="logp", rows=1, vocab=152064, dim=4096, dtype="bf16", k=1,
             masked=0.0, temperature=1.0),
        # serving: a decoding batch with sixteen candidates each
        dict(name="logp_decode_batch", op="logp", rows=48, vocab=32768, dim=2048, dtype="bf16", k=16,
             masked=0.0, temperature=0.9),
        # a rollout's log-probs under the old and reference policies: no gradient, 15% of rows masked
        dict(name="logp_rollout", op="logp", rows=8192, vocab=152064, dim=2560, dtype="bf16", k=4,
             masked=0.15, temperature=0.9),
        # the policy step: log-probs and the gradient an RL loss sends back through them
        dict(name="logp_policy_step", op="logp_step", rows=2048, vocab=151936, dim=2560, dtype="bf16",
             k=1, masked=0.1, temperature=0.9),
        # the same in fp32 at odd sizes
        dict(name="logp_step_fp32_odd", op="logp_step", rows=301, vocab=1003, dim=200, dtype="fp32",
             k=3, masked=0.15, temperature=0.7),
        # ------------------------------------------------ the table's other end
        # decoding: one token of each of 64 sequences
        dict(name="lookup_decode", op="lookup", rows=64, vocab=152064, dim=4096, dtype="bf16",
             ignored=0.0, scale=1.0),
        # the lookup's gradient of a packed step, token frequencies as in text (a few very common)
        dict(name="lookup_grad_packed", op="lookup_grad", rows=8192, vocab=152064, dim=2560,
             dtype="bf16", ignored=0.05, scale=50.5),
        # a tied table's whole gradient: the head's, and the lookup's added to it
        dict(name="tied_step_fp32", op="tied", rows=1024, vocab=32768, dim=1024, dtype="fp32",
             ignored=0.1, temperature=1.0, scale=32.0),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ce", "ce", "logp", "logp", "logp_step", "lookup", "lookup_grad", "tied"])
    dtype = "fp32" if op == "tied" or rng.random() < 0.25 else "bf16"
    big = 2048 if dtype == "fp32" else 8192
    case = dict(op=op, rows=_spread(rng, 1, big), vocab=_spread(rng, 64, 152064),
                dim=_spread(rng, 64, 1024 if dtype == "fp32" else 4096), dtype=dtype)
    if rng.random() < 0.5:  # widths of real models are multiples of 64
        case["dim"] = max(64, case["dim"] // 64 * 64)
    if op in ("ce", "tied", "lookup", "lookup_grad"):
        case["ignored"] = rng.choice([0.0, 0.1, 0.75])
    if op in ("logp", "logp_step"):
        case.update(k=rng.choice([1, 2, 4, 7, 16]), masked=rng.choice([0.0, 0.15, 0.6]))
    if op in ("ce", "tied", "logp", "logp_step"):
        case["temperature"] = rng.choice([1.0, 0.9, 0.7, 1.3])
    if op == "ce":
        case.update(reduction=rng.choice(["mean", "sum", "none"]), pad=rng.choice([0, 0, 5, 8]))
    if op in ("lookup", "lookup_grad", "tied"):
        case["scale"] = rng.choice([1.0, math.sqrt(case["dim"]), 12.0])
    return case


def _table(case, g):
    """Rows of norm about 2.5, so that unit-normal hidden states give logits of std 2.5."""
    std = 2.5 / math.sqrt(case["dim"])
    w = torch.randn((case["vocab"], case["dim"]), generator=g, device="cuda")
    return w.mul_(std).to(DTYPES[case["dtype"]])


def _hidden(case, w, target, g):
    """Unit-normal hidden states; one row in twenty is led by its target (8 to 12 above the others'
    scale) and one in twenty confident far past fp32's 1 - p (margins up to 50)."""
    rows, dim = case["rows"], case["dim"]
    h = torch.randn((rows, dim), generator=g, device="cuda")
    u = torch.rand(rows, generator=g, device="cuda")
    lead = torch.where(u < 0.05, 20.0 + 4.0 * torch.rand(rows, generator=g, device="cuda"),
                       torch.where(u > 0.95, 35.0 + 25.0 * torch.rand(rows, generator=g, device="cuda"),
                                   torch.zeros(rows, device="cuda")))
    wt = w[target].float()
    h += (lead / wt.square().sum(1)).unsqueeze(1) * wt
    pad = int(case.get("pad", 0))
    buf = torch.zeros((rows, dim + pad), dtype=DTYPES[case["dtype"]], device="cuda")
    buf[:, :dim] = h.to(buf.dtype)
    return buf[:, :dim]


def _tokens(case, g, common):
    """Token ids; `common`: as in text, the n-th most common about 1/n as often as the first."""
    rows, vocab = case["rows"], case["vocab"]
    u = torch.rand(rows, generator=g, device="cuda", dtype=torch.float64)
    if common:
        t = torch.exp(u * math.log(vocab + 1.0)).long().sub_(1)
        t = (t * 48271 + 11) % vocab
    else:
        t = (u * vocab).long()
    return t.clamp_(0, vocab - 1)


def _left_out(rows, share, g):
    """Which rows are left out; the first never is."""
    skip = torch.rand(rows, generator=g, device="cuda") < share
    skip[0] = False
    return skip


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    rows, dim, op = case["rows"], case["dim"], case["op"]
    st = dict(op=op, vocab=case["vocab"], temperature=case.get("temperature", 1.0),
              scale=case.get("scale", 1.0), reduction=case.get("reduction", "mean"))
    if op != "lookup_grad":
        st["weight"] = _table(case, g)
    if op in ("ce", "tied"):
        lab = _tokens(case, g, True)
        st["hidden"] = _hidden(case, st["weight"], lab, g)
        skip = _left_out(rows, case["ignored"], g)
        st["labels"] = lab.masked_fill(skip, IGNORE)
        one = {"none": torch.full((rows,), 1.0 / max(1.0, round(rows * (1.0 - case["ignored"])))),
               "sum": torch.full((1,), 1.0 / rows), "mean": torch.ones(1)}[st["reduction"]]
        st["grad_out"] = one.to("cuda")
    if op in ("logp", "logp_step"):
        idx = torch.randint(0, case["vocab"], (rows, case["k"]), generator=g, device="cuda")
        idx[:, 0] = _tokens(case, g, True)
        st["hidden"] = _hidden(case, st["weight"], idx[:, 0], g)
        st["index"] = idx
        st["mask"] = (~_left_out(rows, case["masked"], g)).to(torch.uint8)
        if op == "logp_step":
            st["grad_logp"] = torch.randn((rows, case["k"]), generator=g, device="cuda") / rows
    if op in ("lookup", "lookup_grad", "tied"):
        tok = _tokens(case, g, True)
        skip = _left_out(rows, case["ignored"], g)
        st["tokens"] = tok.masked_fill(skip, IGNORE)
        if op != "lookup":
            st["grad_rows"] = (torch.randn((rows, dim), generator=g, device="cuda")
                               / (rows * st["scale"])).to(DTYPES[case["dtype"]])
    return st


# ----------------------------------------------------------------- plain forms

def _softplus(a):
    return a.clamp(min=0) + torch.log1p(torch.exp(-a.abs()))


def _logsumexp(x, dim):
    m = x.amax(dim, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    return torch.log(torch.exp(x - m).sum(dim)) + m.squeeze(dim)


def _plain_logp(hidden, weight, idx, T):
    """logits / T, log-probs of idx [rows, K] with each column's sum taken over the others, and lse."""
    z = (hidden.float() @ weight.float().t()) / T
    zt = z.gather(1, idx)
    base = _logsumexp(z.scatter(1, idx, -math.inf), 1)            # the columns nobody gathers
    same = idx.unsqueeze(2) == idx.unsqueeze(1)                   # [rows, K, K]
    again = torch.tril(same, -1).any(2)                           # a column gathered before
    drop = same | again.unsqueeze(1)
    part = torch.where(drop, torch.full_like(same, -math.inf, dtype=z.dtype), zt.unsqueeze(1).expand_as(same))
    others = _logsumexp(torch.cat([base[:, None, None].expand(-1, idx.shape[1], 1), part], 2), 2)
    logp = -_softplus(others - zt)
    return z, logp, _logsumexp(z, 1)


def _plain_ce(hidden, weight, labels, grad_out, T, reduction):
    live = labels != IGNORE
    lab = labels.masked_fill(~live, 0).unsqueeze(1)
    z, logp, lse = _plain_logp(hidden, weight, lab, T)
    n = live.sum()
    rows = torch.where(live, -logp[:, 0], torch.zeros_like(lse))
    loss = {"none": rows, "sum": rows.sum(), "mean": rows.sum() / n}[reduction]
    g = grad_out / (n if reduction == "mean" else 1) * live
    dz = torch.exp(z.sub_(lse.unsqueeze(1))).scatter_(1, lab, torch.expm1(logp))
    dz *= (g / T).unsqueeze(1)
    dh = (dz @ weight.float()).to(hidden.dtype)
    return loss, dh, dz.t() @ hidden.float(), n


def _plain_lookup_grad(grad_rows, tokens, scale, vocab):
    live = tokens != IGNORE
    d = torch.zeros((vocab, grad_rows.shape[1]), dtype=torch.float32, device=grad_rows.device)
    return d.index_add_(0, tokens[live], grad_rows[live].float() * scale)


def _plain(st):
    op, T = st["op"], st["temperature"]
    if op in ("ce", "tied"):
        h, w = st["hidden"], st["weight"]
        loss, dh, dw, n = _plain_ce(h, w, st["labels"], st["grad_out"], T, st["reduction"])
        if op == "tied":
            dw += _plain_lookup_grad(st["grad_rows"], st["tokens"], st["scale"], st["vocab"])
        return dict(loss=loss, dhidden=dh, dweight=dw.to(w.dtype), n_items=n)
    if op in ("logp", "logp_step"):
        idx, live = st["index"], st["mask"].bool().unsqueeze(1)
        z, logp, lse = _plain_logp(st["hidden"], st["weight"], idx, T)
        out = dict(logp=torch.where(live, logp, torch.zeros_like(logp)))
        if op == "logp_step":
            g = st["grad_logp"] * live
            same = (idx.unsqueeze(2) == idx.unsqueeze(1)).float()
            gt = (same * g.unsqueeze(1)).sum(2)
            go = ((1.0 - same) * g.unsqueeze(1)).sum(2)
            dz = torch.exp(z.sub_(lse.unsqueeze(1))).mul_(-g.sum(1, keepdim=True))
            dz.scatter_(1, idx, -gt * torch.expm1(logp) - go * torch.exp(logp))
            dz *= 1.0 / T
            out["dhidden"] = (dz @ st["weight"].float()).to(st["hidden"].dtype)
            out["dweight"] = (dz.t() @ st["hidden"].float()).to(st["weight"].dtype)
        return out
    if op == "lookup":
        tok = st["tokens"]
        live = (tok != IGNORE).unsqueeze(1)
        rows = st["weight"][tok.clamp(min=0)].float() * st["scale"]
        return dict(rows=torch.where(live, rows, torch.zeros_like(rows)).to(st["weight"].dtype))
    d = _plain_lookup_grad(st["grad_rows"], st["tokens"], st["scale"], st["vocab"])
    return dict(dtable=d.to(st["grad_rows"].dtype))


def run(st):
    if not own:
        return _plain(st)
    import cross_entropy_gb300 as gbce

    op, T = st["op"], st["temperature"]
    if op in ("ce", "tied"):
        r = gbce.linear_ce_fwd_bwd_fused(st["hidden"], st["weight"], st["labels"], st["grad_out"],
                                         temperature=T, reduction=st["reduction"])
        if op == "tied":
            gbce.embedding_lookup_bwd(st["grad_rows"], st["tokens"], st["vocab"], st["scale"],
                                      dtable=r.dweight, accumulate=True)
        return dict(loss=r.loss, dhidden=r.dhidden, dweight=r.dweight, n_items=r.n_items)
    if op == "logp":
        return dict(logp=gbce.linear_selective_logsoftmax(st["hidden"], st["weight"], st["index"], T,
                                                          st["mask"]))
    if op == "logp_step":
        logp, state = gbce.linear_selective_logsoftmax(st["hidden"], st["weight"], st["index"], T,
                                                       st["mask"], with_state=True)
        dh, dw = gbce.linear_selective_logsoftmax_bwd(st["hidden"], st["weight"], st["index"],
                                                      st["grad_logp"], logp, state, T, st["mask"])
        return dict(logp=logp, dhidden=dh, dweight=dw)
    if op == "lookup":
        return dict(rows=gbce.embedding_lookup(st["weight"], st["tokens"], st["scale"]))
    return dict(dtable=gbce.embedding_lookup_bwd(st["grad_rows"], st["tokens"], st["vocab"],
                                                 st["scale"]))


# ------------------------------------------------------------------ what it costs

def work(case):
    rows, V, D, op = case["rows"], case["vocab"], case["dim"], case["op"]
    e = 2 if case["dtype"] == "bf16" else 4
    live = max(1.0, rows * (1.0 - case.get("ignored", case.get("masked", 0.0))))
    gemm = 2.0 * live * V * D
    if op == "lookup":
        return dict(bytes=2.0 * live * D * e + 8.0 * rows, flops=live * D)
    if op == "lookup_grad":
        return dict(bytes=live * D * e + V * D * e + 8.0 * rows, flops=live * D)
    if op == "logp":
        return dict(bytes=(live * D + V * D) * e + rows * case["k"] * 12.0, flops=gemm)
    # logits, dhidden and dweight: three products; the table read and its gradient written
    if op == "logp_step":
        return dict(bytes=(2.0 * rows * D + 2.0 * V * D) * e + rows * case["k"] * 16.0, flops=3.0 * gemm)
    more = live * D * e if op == "tied" else 0.0
    return dict(bytes=(2.0 * rows * D + 2.0 * V * D) * e + rows * 8.0 + more, flops=3.0 * gemm)


# ---------------------------------------------------------------- 64 bits

def _exact_rows(h, w, idx, T):
    """p [rows, V], and log p of idx with 1 - p taken from the other columns, all in fp64."""
    z = torch.einsum("rd,vd->rv", h, w) / T
    top = z.max(1, keepdim=True).values
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lp, comp = [], []
    for k in range(idx.shape[1]):
        t = idx[:, k:k + 1]
        rest = z.scatter(1, t, -math.inf)
        peak = rest.max(1, keepdim=True).values
        # the others' sum relative to their own largest, so that it never underflows
        away = torch.exp(rest - peak).sum(1, keepdim=True)
        ratio = torch.log(away) + peak - z.gather(1, t)        # log (1 - p) / p
        lp.append(-torch.nn.functional.softplus(ratio, threshold=200.0))
        comp.append(torch.sigmoid(ratio))                       # 1 - p
    return e / total, torch.cat(lp, 1), torch.cat(comp, 1)


def exact(case, seed):
    rows, V, D, op = case["rows"], case["vocab"], case["dim"], case["op"]
    if op not in ("lookup", "lookup_grad") and 6.0 * rows * V * D > 1.0e13:
        return None
    st = prepare(case, seed)
    T = st["temperature"]
    if op == "lookup":
        out = torch.zeros((rows, D), dtype=torch.float64, device="cuda")
        live = st["tokens"] >= 0
        out[live] = st["weight"].double()[st["tokens"][live]] * st["scale"]
        return dict(rows=out)
    dt = None
    if op in ("lookup_grad", "tied"):
        dt = torch.zeros((V, D), dtype=torch.float64, device="cuda")
        live = st["tokens"] >= 0
        dt.index_put_((st["tokens"][live],), st["grad_rows"][live].double() * st["scale"], accumulate=True)
        if op == "lookup_grad":
            return dict(dtable=dt)
    h, w = st["hidden"].double(), st["weight"].double()
    dh = torch.zeros((rows, D), dtype=torch.float64, device="cuda")
    dw = torch.zeros((V, D), dtype=torch.float64, device="cuda") if op != "logp" else None
    token = op in ("ce", "tied")
    live = st["labels"] >= 0 if token else st["mask"] > 0
    n = int(live.sum())
    idx = st["labels"].clamp(min=0).unsqueeze(1) if token else st["index"]
    logp = torch.zeros(idx.shape, dtype=torch.float64, device="cuda")
    if token:
        up = st["grad_out"].double().expand(rows) / (n if st["reduction"] == "mean" else 1)
        up = -up.unsqueeze(1)
    elif op == "logp_step":
        up = st["grad_logp"].double()
    for r in torch.nonzero(live).squeeze(1).split(512):
        p, lp, comp = _exact_rows(h[r], w, idx[r], T)
        logp[r] = lp
        if op == "logp":
            continue
        # d/dz_j of sum_k u_k log p_k = sum_k u_k ([j = t_k] - p_j)
        u = up[r]
        dz = -u.sum(1, keepdim=True) * p
        hit = torch.zeros_like(dz).scatter_add_(1, idx[r], u)
        for k in range(idx.shape[1]):
            t = idx[r][:, k:k + 1]
            mine = hit.gather(1, t)
            dz.scatter_(1, t, mine * comp[:, k:k + 1] - (u.sum(1, keepdim=True) - mine) * p.gather(1, t))
        dz /= T
        dh[r] = dz @ w
        dw += dz.t() @ h[r]
    if op == "logp":
        return dict(logp=logp)
    if op == "logp_step":
        return dict(logp=logp, dhidden=dh, dweight=dw)
    per = -logp[:, 0]
    loss = {"none": per, "sum": per.sum(), "mean": per.sum() / max(n, 1)}[st["reduction"]]
    return dict(loss=loss, dhidden=dh, dweight=dw if dt is None else dw + dt,
                n_items=st["labels"].ge(0).sum())
