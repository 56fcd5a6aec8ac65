"""The post-training losses from their definitions, plain and in 64 bits (torch
on the CPU), and the error bounds the GPU tests allow."""

import math

import torch

NEG = -math.inf
EPS32 = 2.0 ** -24        # half a step of fp32


def logp_rows(x, lab, T):
    """log p of lab [rows] and 1 - p, both from the sum over the other columns."""
    z = x.double() / T
    zy = z.gather(1, lab.unsqueeze(1))
    rest = torch.logsumexp(z.scatter(1, lab.unsqueeze(1), NEG), 1)
    a = rest - zy.squeeze(1)
    return -torch.nn.functional.softplus(a, threshold=700.0), torch.sigmoid(a), z


def log_shares(v):
    """log softmax of a vector, each relative to the largest entry and the sum of the others, so
    that the log of a share near 1 keeps its digits."""
    top = int(v.argmax())
    others = torch.exp(v - v[top])
    others[top] = 0.0
    return (v - v[top]) - torch.log1p(others.sum())


def small_side(lp):
    """min(p, 1 - p) of a distribution given as log p."""
    return torch.minimum(torch.exp(lp), -torch.expm1(lp))


def distill(x, index, teacher, rest, T, mask=None):
    """(loss [rows], dz [rows, V], what fp32 may move a row by: (eps, sum |q - p|, sum w, norm w)).

    A log p or log q carries at most a few roundings of its exponent, about EPS32 times the
    exponents' range, and 8 for the logs and divisions: eps = 4 EPS32 (range + 8).  The largest
    share is 1 - (the others' sum), so it moves by eps (1 - p); every other one by eps p: by
    eps w in all, w = min(p, 1 - p) + min(q, 1 - q)."""
    rows, V = x.shape
    loss = torch.zeros(rows, dtype=torch.float64)
    dz = torch.zeros((rows, V), dtype=torch.float64)
    move = torch.zeros((4, rows), dtype=torch.float64)
    for r in range(rows):
        if mask is not None and not mask[r]:
            continue
        here = index[r] >= 0
        if bool(((index[r] < -1) | (index[r] >= V)).any()):
            loss[r] = dz[r] = math.nan
            continue
        col, inv = torch.unique(index[r][here], return_inverse=True)
        t = teacher[r][here].double() / T
        pr = rest[r].double() if rest is not None else torch.tensor(NEG).double()
        both = torch.cat([t, pr.reshape(1)])
        if bool(torch.isnan(both).any()) or bool((both == math.inf).any()):
            loss[r] = dz[r] = math.nan
            continue
        if both.numel() == 0 or both.max() == NEG:
            continue
        # log p of a column listed more than once: of the sum
        lp = torch.full((col.numel() + 1,), NEG, dtype=torch.float64)
        for c in range(col.numel()):
            lp[c] = torch.logsumexp(t[inv == c], 0)
        lp[-1] = pr
        lp = log_shares(lp)
        p = torch.exp(lp)
        z = x[r].double() / T
        away = z.clone()
        away[col] = NEG
        zr = torch.logsumexp(away, 0)
        lq = log_shares(torch.cat([z[col], zr.reshape(1)]))
        q = torch.exp(lq)
        # p log (p / q) - p + q, a sum of terms >= 0 that cancel nothing
        u = lq - lp
        term = torch.where(u.abs() < 1e-2, p * u * u * (0.5 + u * (1 / 6 + u * (1 / 24 + u * (1 / 120 + u / 720)))),
                           p * (torch.expm1(u) - u))
        loss[r] = torch.where(p > 0, term, q).sum()
        gap = torch.where((lp - lq).abs() < 1.0, p * torch.expm1(lq - lp), q - p)
        gap = torch.where(p > 0, gap, q)
        dz[r] = torch.exp(away - zr) * gap[-1] if zr != NEG else 0.0
        dz[r][col] = gap[:-1]
        eps = 0.0
        for v in (z, both):
            fin = v[torch.isfinite(v)]
            eps += float(fin.max() - fin.min()) if fin.numel() else 0.0
        w = small_side(lp) + small_side(lq)
        move[:, r] = torch.stack([torch.tensor(4 * EPS32 * (eps + 8.0)).double(), gap.abs().sum(), w.sum(), w.norm()])
    return loss, dz, move


def kl_bound(loss, move):
    """What fp32 may move a row's loss by: sum p phi(u) has phi' = e^u - 1, so eps sum |q - p| to
    first order, eps^2 sum w to second, and each p and phi by eps relative."""
    eps, tv, w, _ = move
    return 2.0 * eps * loss.abs() + 2.0 * eps * tv + eps * eps * w


def gap_bound(move):
    """... and its gradient q - p in norm: each side's own error."""
    return move[0] * move[3]


def policy(lp, adv, old, ref, lo, hi, beta):
    """(loss, dloss/dlp) of each row."""
    rho = torch.exp(lp - old) if old is not None else torch.ones_like(lp)
    edge = torch.where(adv > 0, torch.full_like(adv, 1.0 + hi), torch.full_like(adv, 1.0 - lo))
    held = torch.where(adv > 0, rho > edge, rho < edge)
    rho_a = torch.where(adv == 0, torch.zeros_like(adv), rho * adv)
    loss = -torch.where(held & (adv != 0), edge * adv, rho_a)
    d = torch.where(held, torch.zeros_like(adv), -rho_a)
    if beta:
        gap = ref - lp
        loss = loss + beta * (torch.expm1(gap) - gap)
        d = d - beta * torch.expm1(gap)
    return loss, d


def preference(lp, off, ref, live, beta, margin, eps, kind, average):
    """(pair losses, scores, dloss_i/dlp_r [rows], pair of each row or -1)."""
    n = (len(off) - 1) // 2
    rows = lp.numel()
    gap = lp - ref if ref is not None else lp
    score = torch.zeros(2 * n, dtype=torch.float64)
    weight = torch.zeros(rows, dtype=torch.float64)
    seq = torch.full((rows,), -1)
    for s in range(2 * n):
        a, b = int(off[s]), int(off[s + 1])
        keep = live[a:b]
        w = 1.0 / max(1, int(keep.sum())) if average else 1.0
        score[s] = gap[a:b][keep].sum() * w
        weight[a:b][keep] = w
        seq[a:b] = s
    h = score[:n] - score[n:]
    if kind == "squared":
        e = h - 0.5 / beta
        loss, dh = e * e, 2 * e
    else:
        u = beta * (h - margin)
        ls = torch.nn.functional.logsigmoid
        loss = -(1 - eps) * ls(u) - eps * ls(-u)
        dh = beta * (eps * torch.sigmoid(u) - (1 - eps) * torch.sigmoid(-u))
    d = torch.cat([dh, -dh])
    drow = torch.where(seq >= 0, d[seq.clamp(min=0)] * weight, torch.zeros(rows, dtype=torch.float64))
    return loss, score, drow, torch.where(seq >= 0, seq % n, seq)


def softmax_grad(z, lab, comp, g, T):
    """g (p - onehot) / T per row, 1 - p of the label given."""
    d = torch.softmax(z, 1)
    d.scatter_(1, lab.unsqueeze(1), -comp.unsqueeze(1))
    return d * (g / T).unsqueeze(1)
