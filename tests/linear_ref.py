"""The calls that start from hidden states, in 64 bits and in their plainest
form, with bounds on what an fp32 (or bf16) evaluation may be off by.

Bounds.  u = 2^-24.  A logit is a sum of dim products; dim / 8 + 16 half ulps
of sum |h w| cover a blocked or random-walk fp32 accumulation (and, for fp32
inputs split into three bf16 parts, the dropped products, each below u |h w|),
so z carries at most
    ez = (dim / 8 + 16) u max_v sum_d |h w| / T.
* log p = -softplus(a), a = log(others / e^z_t): |da| <= 2 ez + the roundings
  of a (|a| <= |log p| + 64 for margins up to 64: 2 u of it), so
    |d log p| <= (1 - p) (2 ez + 2 u (|log p| + 64)) + 4 u |log p|.
* dlogits: p carries 2 ez + 16 u relative (exp2, 1 / S, the coefficient), then
  in a bf16 call one rounding, eps/2 = 2^-8.
  Worst case over the products: each sum is off by at most
    (2 ez + 16 u + half step + (n / 8 + 16) u) * sum |dz| |other factor|
  plus its output's own rounding, half a step of |value|.
The half step of a type is finfo.eps / 2 (2^-8 for bf16, 2^-24 for fp32).
"""

import math

import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def rows_of(hidden, weight, targets, T, live):
    """p, log p of the targets, 1 - p of them, and ez, for the live rows (fp64)."""
    h, w = hidden[live].double(), weight.double()
    z = h @ w.t() / T
    ez = ((h.shape[1] / 8 + 16) * U / T * (h.abs() @ w.abs().t())).amax(1, keepdim=True)
    t = targets[live]
    safe = t.clamp(0, w.shape[0] - 1)
    logp = torch.empty(t.shape, dtype=torch.float64, device=h.device)
    comp = torch.empty_like(logp)
    for k in range(t.shape[1]):
        rest = z.scatter(1, safe[:, k:k + 1], -math.inf)
        m = rest.amax(1, keepdim=True)
        if w.shape[0] == 1:
            a = torch.full_like(m, -math.inf)
        else:
            a = torch.exp(rest - m).sum(1, keepdim=True).log() + m - z.gather(1, safe[:, k:k + 1])
        logp[:, k] = -torch.nn.functional.softplus(a, threshold=200.0)[:, 0]
        comp[:, k] = torch.sigmoid(a)[:, 0]
    bad = (t < 0) | (t >= w.shape[0])
    logp[bad] = math.nan
    return torch.softmax(z, 1), logp, comp, ez


def logp_bound(logp, comp, ez):
    return comp * (2 * ez + 2 * U * (logp.abs() + 64)) + 4 * U * logp.abs() + 2.0 ** -148


def selective_dz(p, logp, comp, targets, g, T):
    """dL/dz of sum_k g_k log p_k."""
    hit = torch.zeros_like(p).scatter_add_(1, targets, g)
    total = g.sum(1, keepdim=True)
    dz = -total * p
    size = total.abs() * p
    for k in range(targets.shape[1]):
        t = targets[:, k:k + 1]
        same = targets == t
        mine = hit.gather(1, t)
        other = torch.where(same, torch.zeros_like(g), g).sum(1, keepdim=True)
        dz.scatter_(1, t, mine * comp[:, k:k + 1] - other * p.gather(1, t))
        # the two terms may cancel: what each may be off by counts
        size.scatter_(1, t, g.abs().sum(1, keepdim=True) * (comp[:, k:k + 1] + p.gather(1, t)))
    return dz / T, size / T


def products(dz, size, h, w, ez, dtype):
    """dhidden and dweight of the live rows and their bounds."""
    rel = 2 * ez + 16 * U
    dz_off = size * rel + (dz.abs() + size * rel) * (HALF[dtype] if dtype != torch.float32 else 4 * U)
    dh, dw = dz @ w, dz.t() @ h
    dh_b = dz_off @ w.abs() + (w.shape[0] / 8 + 16) * U * (dz.abs() @ w.abs())
    dw_b = dz_off.t() @ h.abs() + (h.shape[0] / 8 + 16) * U * (dz.abs().t() @ h.abs())
    return dh, dw, dh_b * 1.01 + HALF[dtype] * dh.abs() + 1e-36, \
        dw_b * 1.01 + HALF[dtype] * dw.abs() + 1e-36


def assert_within(got, ref, bound, what):
    got, ref = got.double(), ref.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN pattern differs"
    ok = ~torch.isnan(ref)
    off = (got - ref).abs()[ok] - bound.expand_as(ref)[ok]
    if off.numel():
        worst = int(off.argmax())
        assert off[worst] <= 0, (f"{what}: off by {(got - ref).abs()[ok][worst]:.3e}, bound "
                                 f"{bound.expand_as(ref)[ok][worst]:.3e}, value {ref[ok][worst]:.3e}")
