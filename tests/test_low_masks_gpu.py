"""Vocabularies masked with the type's lowest value, or another far below what the exponentials
span: as if masked with -inf, in the log-probs, the cross-entropies, the entropy and every gradient."""

import pytest
import torch

from helpers import GRAD_FLOOR, GRAD_TOL, LOGP_TOL

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import cross_entropy_gb300 as gbce

DEV = "cuda:0"
NEG, NAN = float("-inf"), float("nan")
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__

    __graft_entry__.build()
    gbce.load_library()


# split rows, short and long ones, more of them than CTAs
PLACES = [(8, 5, F32), (8, 300, BF16), (8, 5000, F32), (8, 152064, BF16), (8, 100001, F32), (500, 40001, BF16),
          (1300, 20000, F32), (2000, 4099, BF16)]
LOOKED_AT = 8


def masked(rows, V, dtype, seed):
    """Logits, which columns are kept (a random tenth, the label alone, the last half, the first half, one
    vector, everything, a tenth, a quarter), the label and a second column."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = (torch.randn((rows, V), generator=g, device=DEV) * 2.0).to(dtype)
    keep = torch.rand((rows, V), generator=g, device=DEV) < 0.1
    keep[1] = False
    keep[2], keep[3] = False, False
    keep[2, V // 2:] = True
    keep[3, :V // 2] = True
    keep[4] = False
    keep[4, V // 3:V // 3 + 8] = True
    keep[5] = True
    keep[7] = torch.rand(V, generator=g, device=DEV) < 0.25
    idx = torch.randint(0, V, (rows, 2), generator=g, device=DEV)
    keep.scatter_(1, idx[:, :1], True)
    return x, keep, idx


def norms_close(got, want, dtype, what):
    """Each row's gradient in norm, with its type's rounding floor."""
    got, want = got.double(), want.double()
    off = (got - want).norm(dim=1)
    bound = GRAD_TOL[dtype] * want.norm(dim=1) + GRAD_FLOOR[dtype] * want.shape[1] ** 0.5
    assert bool((off <= bound).all()), (what, (off - bound).max())


@pytest.mark.parametrize("fill", [None, -1e30, -1e12, -1e9])
@pytest.mark.parametrize("T", [1.0, 0.7])
@pytest.mark.parametrize("rows,V,dtype", PLACES)
def test_as_if_masked_with_minus_infinity(rows, V, dtype, T, fill):
    x, keep, idx = masked(rows, V, dtype, V)
    y = x.masked_fill(~keep, torch.finfo(dtype).min if fill is None else fill)
    n = LOOKED_AT
    z = (x[:n].double() / T).masked_fill(~keep[:n], NEG)
    p = torch.softmax(z, 1)
    lab = idx[:, 0].contiguous()
    # log p from the others' sum, as an exact one near 0 needs
    rest = torch.logsumexp(z.scatter(1, idx[:n, :1], NEG), 1)
    lp = -torch.nn.functional.softplus(rest - z.gather(1, idx[:n, :1])[:, 0], threshold=700.0)
    dz = p.scatter(1, idx[:n, :1], torch.expm1(lp).unsqueeze(1)) / T
    ent = -torch.where(p > 0, p * torch.log_softmax(z, 1), torch.zeros_like(p)).sum(1)
    one = torch.ones(rows, device=DEV)

    def logp_close(got, what):
        off = (got[:n].double() - lp).abs() - LOGP_TOL[dtype] * lp.abs() - 2.0 ** -148
        assert bool((off <= 0).all()), (what, off)
        assert bool(torch.isfinite(got).all()), what

    sel = gbce.selective_logsoftmax(y, lab, T)
    logp_close(sel, "selective")
    both, H = gbce.selective_logsoftmax(y, lab, T, with_entropy=True)
    logp_close(both, "with entropy")
    assert bool(((H[:n].double() - ent).abs() <= 2e-5 * ent + 1e-30).all()), (H[:n], ent)
    two = gbce.selective_logsoftmax(y, idx, T)
    logp_close(two[:, 0], "two columns")
    f = gbce.ce_fwd(y, lab, temperature=T, reduction="none")
    logp_close(-f.loss, "ce")
    u = gbce.ce_fwd_bwd_fused(y, lab, one, temperature=T, reduction="none")
    logp_close(-u.loss, "fused ce")
    v = gbce.ce_fwd_bwd_fused_noalloc(y, lab, one, temperature=T, reduction="none")
    logp_close(-v.loss, "noalloc")
    b = gbce.ce_bwd(y, lab, one, f.logp, temperature=T, reduction="none")
    s = gbce.selective_logsoftmax_bwd(y, lab, -one, sel, T)
    for what, d in (("fused", u.dlogits), ("noalloc", v.dlogits), ("ce_bwd", b), ("selective_bwd", s)):
        norms_close(d[:n], dz, dtype, what)
        assert bool(torch.isfinite(d).all()), what
    e = gbce.selective_logsoftmax_bwd(y, lab, -one, sel, T, grad_entropy=one, saved_entropy=H)
    dH = -p * (torch.where(p > 0, torch.log_softmax(z, 1), torch.zeros_like(p)) + ent.unsqueeze(1)) / T
    norms_close(e[:n], dz + dH, dtype, "with the entropy's gradient")


@pytest.mark.parametrize("rows,V,dtype", PLACES)
def test_a_masked_label_and_a_row_of_masks(rows, V, dtype):
    """A label at the lowest value beside others: log p as low, the gradient the others' softmax.  A row
    at the lowest value throughout has no log p."""
    x, keep, idx = masked(rows, V, dtype, V + 1)
    low = torch.finfo(dtype).min
    lab = idx[:, 0].contiguous()
    x[0, lab[0]] = low
    x[1] = low
    one = torch.ones(rows, device=DEV)
    want = torch.softmax(x[0].double(), 0)
    want[lab[0]] = -1.0
    sel, H = gbce.selective_logsoftmax(x, lab, with_entropy=True)
    u = gbce.ce_fwd_bwd_fused(x, lab, one, reduction="none")
    s = gbce.selective_logsoftmax_bwd(x, lab, -one, gbce.selective_logsoftmax(x, lab))
    assert float(sel[0]) < -3e38 and float(u.loss[0]) > 3e38 and bool(torch.isfinite(H[0]))
    norms_close(u.dlogits[:1], want.unsqueeze(0), dtype, "fused")
    norms_close(s[:1], want.unsqueeze(0), dtype, "selective")
    for v in (sel[1], H[1], u.loss[1]):
        assert bool(torch.isnan(v))
    rest = torch.ones(rows, dtype=torch.bool, device=DEV)
    rest[:2] = False
    assert bool(torch.isfinite(sel[rest]).all()) and bool(torch.isfinite(u.dlogits[rest]).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_slices_that_are_masked_out(dtype):
    """A vocabulary in slices, some of which are masked throughout for a row."""
    rows, V, cuts = 9, 12000, [0, 3000, 3500, 9000, 12000]
    g = torch.Generator(device=DEV).manual_seed(3)
    x = (torch.randn((rows, V), generator=g, device=DEV) * 2.0).to(dtype)
    keep = torch.zeros((rows, V), dtype=torch.bool, device=DEV)
    for r in range(rows):
        keep[r, cuts[r % 4]:cuts[r % 4 + 1]] = True
    keep[8] = True
    idx = torch.tensor([[cuts[r % 4] + 7] for r in range(rows)], device=DEV)
    y = x.masked_fill(~keep, torch.finfo(dtype).min)
    z = x.double().masked_fill(~keep, NEG)
    want = torch.log_softmax(z, 1).gather(1, idx)
    parts = [gbce.vocab_slice_stats(y[:, a:b], idx, a, V) for a, b in zip(cuts, cuts[1:])]
    logp, xt, state = gbce.vocab_slice_combine(torch.stack(parts), cuts, idx)
    assert bool(((logp.double().view(rows, 1) - want).abs() <= LOGP_TOL[dtype] * want.abs()).all())
    one = torch.ones(rows, device=DEV)
    d = torch.cat([gbce.vocab_slice_grad(y[:, a:b], idx, a, V, one, logp, xt, row_state=state)
                   for a, b in zip(cuts, cuts[1:])], 1)
    norms_close(d, -torch.softmax(z, 1).scatter(1, idx, torch.expm1(want)), dtype, "slices")


@pytest.mark.parametrize("rows,V,dtype", PLACES + [(8, 2, F32), (8, 2, BF16), (8, 4097, F32), (8, 1025, F32),
                                                   (8, 257, BF16), (2000, 4105, BF16)])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_one_nan_wherever_it_lies(rows, V, dtype, shift):
    """A NaN logit makes its row NaN: at either end, and between columns that are all -inf."""
    g = torch.Generator(device=DEV).manual_seed(V + shift)
    buf = torch.zeros(rows * (V + shift) + shift, dtype=dtype, device=DEV)
    x = buf[shift:].view(rows, V + shift)[:, :V]
    x.copy_(torch.randn((rows, V), generator=g, device=DEV) * 2.0)
    lab = torch.ones(rows, dtype=torch.int64, device=DEV)
    lab[1] = 0
    at = [(0, 0), (1, V - 1)]
    if V > 64:
        x[3:6] = NEG
        x[3:6, 1] = 1.0
        at += [(3, V // 2), (4, V - 1), (5, 40)]
    for r, c in at:
        x[r, c] = NAN
    bad = torch.zeros(rows, dtype=torch.bool, device=DEV)
    bad[[r for r, _ in at]] = True
    one = torch.ones(rows, device=DEV)
    idx = torch.stack([lab, 1 - lab], 1)
    sel, H = gbce.selective_logsoftmax(x, lab, with_entropy=True)
    two, H2 = gbce.selective_logsoftmax(x, idx, with_entropy=True)
    f = gbce.ce_fwd(x, lab, reduction="none")
    c = gbce.ce_fwd(x, lab, reduction="none", softcap=30.0)
    u = gbce.ce_fwd_bwd_fused(x, lab, one, reduction="none")
    n = gbce.ce_fwd_bwd_fused_noalloc(x, lab, one, reduction="none")
    only = gbce.selective_logsoftmax(x, lab)
    b = gbce.ce_bwd(x, lab, one, f.logp, reduction="none")
    s = gbce.selective_logsoftmax_bwd(x, lab, one, only)
    for name, v in dict(sel=sel, H=H, H2=H2, two=two[:, 0], ce=f.loss, cap=c.loss, fused=u.loss, noalloc=n.loss,
                        only=only).items():
        assert torch.equal(torch.isnan(v), bad), name
    for name, d in dict(fused=u.dlogits, noalloc=n.dlogits, ce_bwd=b, selective_bwd=s).items():
        assert torch.equal(torch.isnan(d).all(1), bad) and torch.equal(torch.isnan(d).any(1), bad), name
    if shift == 0 and V > 64:
        cuts = [0, V // 3, V // 2, V]
        parts = [gbce.vocab_slice_stats(x[:, i:j], lab, i, V) for i, j in zip(cuts, cuts[1:])]
        assert torch.equal(torch.isnan(gbce.vocab_slice_combine(torch.stack(parts), cuts, lab.view(-1, 1))[0]).view(-1), bad)


@pytest.mark.parametrize("rows,V,dtype", PLACES)
def test_logits_far_from_zero_at_a_low_temperature(rows, V, dtype):
    """x / T of -1.34e9 to -1.48e9: x c above -2^31, so every row keeps its log p.  (Below it the shift's
    half step is 128, and 2^-128 is not a normal number: some rows' sums are 0, and their log p NaN.)"""
    g = torch.Generator(device=DEV).manual_seed(V + 5)
    T = 2.0 ** -26
    x = (-22.0 + 2.0 * torch.rand((rows, V), generator=g, device=DEV)).to(dtype)
    lab = torch.randint(0, V, (rows,), generator=g, device=DEV)
    x[0, lab[0]] = -19.0
    z = x.double() / T
    want = torch.log_softmax(z, 1).gather(1, lab.unsqueeze(1))[:, 0]
    for got in (gbce.selective_logsoftmax(x, lab, T), -gbce.ce_fwd(x, lab, temperature=T, reduction="none").loss):
        assert bool(((got.double() - want).abs() <= LOGP_TOL[dtype] * want.abs() + 1e-30).all())
