"""Edges of the post-training losses: many rows whose loss the warps of a CTA sum together, masks of the
type's lowest value, NaN beside -inf, labels and offsets that are no use."""

import math

import pytest
import torch

import post_ref as ref
import test_post_gpu as base
from test_post_gpu import BF16, DEV, F32, IGNORE, INF, NAN, NEG, gbce, gen, gpu, logits_of, teacher_of  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,V,K,dtype", [(4000, 5000, 33, BF16), (4000, 9000, 64, BF16), (3000, 3000, 256, F32),
                                            (2000, 30000, 100, BF16), (1500, 14000, 256, F32)])
def test_forward_of_many_listed_entries(gbce, rows, V, K, dtype):  # noqa: F811
    """Warps that share a row finish it at different times (four and eight of them, some without entries):
    every row's state is its own max and sum, the loss the fused call's and the definition's, and all of
    it the same bits each time.  (A sum's terms carry the rounding of their exponents, which span some 30,
    and of 2^x: 30 2^-24 + 2^-22 = 2e-6.  The losses are 3 or more, as 1 to 3% of the columns are listed;
    four roundings of log p and log q each, over a range of 30, move them by 2 * 9e-6 (KL + 2) at most.)"""
    g = torch.Generator(device=DEV).manual_seed(V + K)
    x = (torch.randn((rows, V), generator=g, device=DEV) * 2.0).to(dtype)
    width = V // K
    idx = torch.randint(0, width, (rows, K), generator=g, device=DEV) + torch.arange(K, device=DEV) * width
    t = x.float().gather(1, idx) + torch.randn((rows, K), generator=g, device=DEV)
    first = gbce.distill_fwd(x, idx, t, None, 1.0, None, "none")
    z = x.double().scatter(1, idx, NEG)
    m = z.max(1, keepdim=True).values
    s = torch.exp(z - m).sum(1)
    del z
    assert torch.equal(first.rest_state[:, 0].double(), m[:, 0])
    assert float((first.rest_state[:, 1].double() / s - 1).abs().max()) <= 2e-5
    logp = torch.log_softmax(t.double(), 1)
    lse = torch.logsumexp(x.double(), 1, keepdim=True)
    kl = (torch.exp(logp) * (logp - (x.double().gather(1, idx) - lse))).sum(1)
    one = torch.ones(rows, device=DEV)
    fused = gbce.distill_fwd_bwd_fused(x, idx, t, None, one, 1.0, None, "none")
    for loss in (first.loss, fused.loss):
        assert float(((loss.double() - kl).abs() / (kl + 1e-2)).max()) <= 1e-4
    for _ in range(100):
        again = gbce.distill_fwd(x, idx, t, None, 1.0, None, "none")
        assert torch.equal(again.loss, first.loss) and torch.equal(again.rest_state, first.rest_state)


def test_squared_preference_takes_no_notice_of_the_sigmoids_options(gbce):  # noqa: F811
    """One set of options serves both kinds: the squared loss has neither a margin nor smoothing."""
    g = gen(5)
    x, lab = gpu(logits_of(12, 90, F32, g)), gpu(torch.randint(0, 90, (12,), generator=g))
    off = [0, 3, 6, 9, 12]
    want = gbce.preference_loss_fwd_bwd_fused(x, lab, off, kind="squared", beta=0.5)
    got = gbce.preference_loss_fwd_bwd_fused(x, lab, off, kind="squared", beta=0.5, margin=0.5, label_smoothing=0.1)
    assert torch.equal(got.loss, want.loss) and torch.equal(got.dlogits, want.dlogits)
    one = gbce.preference_loss(want.logp, off, kind="squared", beta=0.5, margin=0.5, label_smoothing=0.1)
    two = gbce.preference_loss(want.logp, off, kind="squared", beta=0.5)
    assert torch.equal(one.loss, two.loss) and torch.equal(one.dlogp, two.dlogp)
    # in effect for the other kind
    assert not torch.equal(gbce.preference_loss(want.logp, off, margin=0.5).loss,
                           gbce.preference_loss(want.logp, off).loss)


# rows, V, dtype, where they go: one, four, eight warps a row; split over a cluster; streamed, by CTAs of
# each shape
PLACES = [(402, 300, F32), (402, 4001, BF16), (9, 3001, F32), (20, 30000, BF16), (20, 20001, F32), (9, 60001, BF16),
          (9, 30001, F32), (240, 60001, BF16), (600, 30001, F32), (500, 100000, BF16), (460, 50001, F32)]
SPECIAL = 8   # rows that are looked at


def masked_rows(rows, V, dtype, fill, K, g):
    """Logits with masked columns at `fill`, the same with -inf there, labels, teacher columns: a random
    quarter, a tenth, the first half, the last half, all but the label or the entries, everything (no
    -inf: all columns alike), nothing, a single vector kept."""
    x = torch.full((rows, V), 0.0)
    x[:SPECIAL] = torch.randn((SPECIAL, V), generator=g) * 2.0
    keep = torch.rand((SPECIAL, V), generator=g) < torch.tensor([0.25, 0.1, 1, 1, 0, 0, 1, 0]).unsqueeze(1)
    keep[2, V // 2:] = False
    keep[3, :V // 2] = False
    keep[7, 40:48] = True
    lab = torch.randint(0, V, (rows,), generator=g)
    lab[2], lab[3], lab[7] = 5, V - 1, 44
    idx = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(rows)])
    for r in range(SPECIAL):
        if r != 5:
            keep[r, lab[r]] = True
    x = x.to(dtype)
    low = fill if fill is not None else torch.finfo(dtype).min
    far, gone = x.clone(), x.clone()
    far[:SPECIAL][~keep] = low
    gone[:SPECIAL][~keep] = NEG
    gone[5] = 0.0
    return far, gone, keep, lab, idx


@pytest.mark.parametrize("fill,T", [(None, 1.0), (None, 0.7), (None, 2.0), (-1e9, 1.0), (-1e4, 0.7), (-1e30, 1.3)])
@pytest.mark.parametrize("rows,V,dtype", PLACES)
def test_masks_of_a_low_value(gbce, rows, V, dtype, fill, T):  # noqa: F811
    """A masked column has no mass whatever low value it holds, and columns that all hold one share it.
    (At -1e4 and -1e9 the masks' shares underflow too; the reference has -inf there.)"""
    g = gen(V + 7)
    far, gone, keep, lab, _ = masked_rows(rows, V, dtype, fill, 4, g)
    n = SPECIAL
    lp, comp, z = ref.logp_rows(gone[:n].float(), lab[:n], T)
    adv = torch.rand(rows, generator=g) + 0.5
    one = torch.ones(rows, device=DEV)
    xg, labg = gpu(far), gpu(lab)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    p = gbce.policy_loss_fwd_bwd_fused(xg, labg, gpu(adv), None, None, one, reduction="none", temperature=T,
                                       dev_status=flag)
    base.close(p.logp[:n], lp, base.LOGP_TOL[dtype], 2.0 ** -148, "policy logp")
    base.rows_close(p.dlogits[:n], ref.softmax_grad(z, lab[:n], comp, adv[:n].double(), T), dtype, "policy")
    off = torch.tensor([0, rows // 2, rows])
    q = gbce.preference_loss_fwd_bwd_fused(xg, labg, gpu(off), temperature=T, average=True, dev_status=flag)
    base.close(q.logp[:n], lp, base.LOGP_TOL[dtype], 2.0 ** -148, "preference logp")
    h = float(q.seq_score[0] - q.seq_score[1])
    drow = torch.full((n,), -0.1 / (1 + math.exp(0.1 * h)) / (rows // 2)).double()
    if n > rows // 2:
        drow[rows // 2:] *= -(rows // 2) / (rows - rows // 2)
    base.rows_close(q.dlogits[:n], ref.softmax_grad(z, lab[:n], comp, -drow, T), dtype, "preference",
                    1e-6 * drow.abs())
    assert int(flag) == 0


@pytest.mark.parametrize("fill,T", [(None, 1.0), (None, 0.7), (-1e9, 1.0), (-1e30, 1.3)])
@pytest.mark.parametrize("rows,V,dtype", PLACES)
def test_distill_over_masks_of_a_low_value(gbce, rows, V, dtype, fill, T):  # noqa: F811
    """... where the teacher's list holds masked columns too, its own logits there just as low."""
    g = gen(V + 8)
    K = 40
    far, gone, keep, lab, idx = masked_rows(rows, V, dtype, fill, K, g)
    n = SPECIAL
    idx[:n, 0] = lab[:n]
    for r in range(n):                       # (the label stays the only one of its columns)
        idx[r, 1:][idx[r, 1:] == lab[r]] = -1
    t = far.float().gather(1, idx.clamp(min=0)) + 0.7 * torch.randn((rows, K), generator=g)
    t[:, 0] = far.float().gather(1, lab.unsqueeze(1))[:, 0].clamp(min=-9.0) + 1.0
    seen = t.clone()
    here = torch.zeros((rows, K), dtype=torch.bool)
    here[:n] = keep.gather(1, idx[:n].clamp(min=0))
    here[5] = True
    seen[:n] = t[:n].masked_fill(~here[:n], NEG)
    t[:n] = torch.where(here[:n], t[:n], torch.full_like(t[:n], -3e38 if fill is None else fill))
    t[5], seen[5] = 0.5, 0.5
    per, dz, move = ref.distill(gone[:n].float(), idx[:n], seen[:n], None, T)
    one = torch.ones(rows, device=DEV)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = (gpu(far), gpu(idx), gpu(t), None)
    out = gbce.distill_fwd_bwd_fused(*args, one, T, None, "none", dev_status=flag)
    f = gbce.distill_fwd(*args, T, None, "none", dev_status=flag)
    b = gbce.distill_bwd(*args, one, f.rest_state, None, T, None, "none", dev_status=flag)
    assert int(flag) == 0
    for what, loss, d in (("fused", out.loss, out.dlogits), ("two calls", f.loss, b)):
        base.close(loss[:n], per, base.LOSS_TOL, ref.kl_bound(per, move).nan_to_num(0.0, 0.0, 0.0), what)
        base.rows_close(d[:n], dz / T, dtype, what, ref.gap_bound(move) / T)


@pytest.mark.parametrize("rows,V,dtype", PLACES)
def test_a_masked_label(gbce, rows, V, dtype):  # noqa: F811
    """A label at the type's lowest value beside others that are not: log p as low, and no NaN."""
    g = gen(V + 9)
    x = torch.zeros((rows, V), dtype=dtype)
    x[:2] = (torch.randn((2, V), generator=g) * 2.0).to(dtype)
    lab = torch.randint(0, V, (rows,), generator=g)
    x[0, lab[0]] = torch.finfo(dtype).min
    one = torch.ones(rows, device=DEV)
    p = gbce.policy_loss_fwd_bwd_fused(gpu(x), gpu(lab), one, one * -2.0, None, one, reduction="none")
    assert float(p.logp[0]) < -3e38 and float(p.loss[0]) == 0 and not bool(p.dlogits[0].any())
    assert bool(torch.isfinite(p.loss[1:]).all()) and bool(torch.isfinite(p.dlogits).all())


@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("rows,V,dtype", PLACES + [(3, 2, BF16), (402, 2, F32), (6, 4097, F32), (402, 1025, F32),
                                                   (402, 257, BF16), (7, 4105, BF16)])
def test_one_nan_wherever_it_lies(gbce, rows, V, dtype, shift):  # noqa: F811
    """A NaN logit makes its row NaN: at either end, and between columns that are all -inf."""
    g = gen(V + 10 + shift)
    x = torch.zeros((rows, V), dtype=dtype)
    x[:6] = (torch.randn((min(rows, 6), V), generator=g) * 2.0).to(dtype)
    at = [(0, 0), (1, V - 1)]
    lab = torch.ones(rows, dtype=torch.int64)
    lab[1] = 0
    if V > 64:
        x[3], x[4], x[5] = NEG, NEG, NEG
        for r in (3, 4, 5):
            x[r, 1] = 1.0
        at += [(3, V // 2), (4, V - 1), (5, 40)]
    for r, c in at:
        x[r, c] = NAN
    n = min(rows, 7)
    bad = torch.zeros(n, dtype=torch.bool)
    bad[[r for r, _ in at]] = True
    one = torch.ones(rows, device=DEV)
    xg = base.on_gpu(x, shift, shift)
    p = gbce.policy_loss_fwd_bwd_fused(xg, gpu(lab), one, None, None, one, reduction="none")
    q = gbce.preference_loss_fwd_bwd_fused(xg, gpu(lab), [0, rows, rows], reduction="sum")
    idx = lab.unsqueeze(1)
    t = torch.zeros((rows, 1))
    d = gbce.distill_fwd_bwd_fused(xg, gpu(idx), gpu(t), None, one, 1.0, None, "none")
    f = gbce.distill_fwd(xg, gpu(idx), gpu(t), None, 1.0, None, "none")
    b = gbce.distill_bwd(xg, gpu(idx), gpu(t), None, one, f.rest_state, None, 1.0, None, "none")
    for v in (p.loss, p.logp, q.logp, d.loss, f.loss):
        assert torch.equal(torch.isnan(v[:n]).cpu(), bad), v[:n]
    for v in (p.dlogits, d.dlogits, b):
        assert torch.equal(torch.isnan(v[:n]).all(1).cpu(), bad) and torch.equal(torch.isnan(v[:n]).any(1).cpu(), bad)
    assert bool(torch.isnan(q.loss)) and bool(torch.isnan(q.dlogits).all())


BAD_OFFSETS = [[0, 2, 10, 5, 7], [0, 6, 3, 9, 12], [0, 3, 6, 9, 13], [-1, 3, 6, 9, 12], [0, 3, 1 << 40, 9, 12],
               [0, 1, 5, 6, 10, 3, 4, 8, 12], [0, 8, 2, 3, 4, 9, 12], [2, 4, 11, 10, 11], [12, 8, 6, 4, 0], [5, 9, 1, 2, 3]]


@pytest.mark.parametrize("off", BAD_OFFSETS)
@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_offsets_that_are_no_use(gbce, off, reduction):  # noqa: F811
    """Offsets that go down anywhere, or leave the rows: no pair keeps a loss, a score or a gradient."""
    g = gen(31)
    rows, pairs = 12, (len(off) - 1) // 2
    x = gpu(logits_of(rows, 90, F32, g))
    lab = torch.randint(0, 90, (rows,), generator=g)
    lab[4] = IGNORE
    mask = (lab != IGNORE).to(torch.uint8)
    inside = (torch.arange(rows) >= max(off[0], 0)) & (torch.arange(rows) < min(off[-1], rows)) & (lab != IGNORE)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    opt = dict(reduction=reduction, dev_status=flag)
    out = gbce.preference_loss_fwd_bwd_fused(x, gpu(lab), off, **opt,
                                             grad_out=torch.ones(pairs if reduction == "none" else 1))
    assert int(flag) == 2
    flag.zero_()
    two = gbce.preference_loss(torch.full((rows,), -1.0, device=DEV), off, None,
                               torch.ones(pairs if reduction == "none" else 1), gpu(mask), **opt)
    assert int(flag) == 2
    for r in (out, two):
        assert bool(torch.isnan(r.loss).all()) and bool(torch.isnan(r.seq_score).all())
    for d in (out.dlogits, two.dlogp.view(rows, 1)):
        assert torch.equal(torch.isnan(d).any(1).cpu(), inside) and torch.equal(torch.isnan(d).all(1).cpu(), inside)
        assert not bool(d[gpu(~inside)].any())


@pytest.mark.parametrize("rows,V,dtype", PLACES)
def test_rows_that_have_no_softmax(gbce, rows, V, dtype):  # noqa: F811
    """A label of +inf, another column of +inf, a row of -inf throughout: NaN, in every loss.  A label
    that alone is not -inf is certain."""
    g = gen(V + 11)
    x = torch.zeros((rows, V), dtype=dtype)
    x[:6] = (torch.randn((6, V), generator=g) * 2.0).to(dtype)
    lab = torch.randint(0, V, (rows,), generator=g)
    x[0, lab[0]] = INF
    x[1, (lab[1] + 1) % V] = INF
    x[2] = NEG
    x[3] = NEG
    x[3, lab[3]] = 1.0
    bad = torch.tensor([True, True, True, False, False, False])
    one = torch.ones(rows, device=DEV)
    xg, idx, t = gpu(x), gpu(lab.unsqueeze(1)), torch.zeros((rows, 1), device=DEV)
    p = gbce.policy_loss_fwd_bwd_fused(xg, gpu(lab), one, None, None, one, reduction="none")
    off = [0, 1, 2, 3, 4, 5, 6, 6, rows]       # six sequences of a row, an empty one, the rest
    q = gbce.preference_loss_fwd_bwd_fused(xg, gpu(lab), off, reduction="none")
    d = gbce.distill_fwd_bwd_fused(xg, idx, t, None, one, 1.0, None, "none")
    f = gbce.distill_fwd(xg, idx, t, None, 1.0, None, "none")
    b = gbce.distill_bwd(xg, idx, t, None, one, f.rest_state, None, 1.0, None, "none")
    for v in (p.loss, p.logp, q.logp, q.seq_score, d.loss, f.loss):
        assert torch.equal(torch.isnan(v[:6]).cpu(), bad), v[:6]
    for v in (p.dlogits, d.dlogits, b):
        assert torch.equal(torch.isnan(v[:6]).all(1).cpu(), bad) and torch.equal(torch.isnan(v[:6]).any(1).cpu(), bad)
    for v in (p.logp, p.loss + 1.0, q.logp, d.loss, f.loss):
        assert float(v[3]) == 0.0
    for v in (p.dlogits, d.dlogits, b):
        assert not bool(v[3].any())
    # pair i holds sequences i and 4 + i
    assert torch.isnan(q.loss).tolist() == [True, True, True, False]
    assert torch.isnan(q.dlogits[:6]).all(1).tolist() == [True] * 3 + [False] + [True] * 2


@pytest.mark.parametrize("eps", [0.0, 0.1])
def test_smoothing_beside_an_infinite_score(gbce, eps):  # noqa: F811
    """An answer that the policy cannot give has log p -inf: the loss of its pair is +inf where it was
    chosen, and eps times that where it was rejected; the slope stays (1 - eps) beta and eps beta."""
    lp = torch.tensor([-1.0, NEG, -2.0, -1.0, -1.0, -3.0, NEG, -0.5])
    off = [0, 2, 4, 6, 8]                      # pair 0: chosen -inf; pair 1: rejected -inf
    r = gbce.preference_loss(gpu(lp), off, label_smoothing=eps, reduction="none", grad_out=torch.ones(2), beta=0.5)
    assert r.loss.tolist() == [INF, INF if eps else 0.0]
    want = torch.tensor([-(1 - eps), eps, 1 - eps, -eps]).repeat_interleave(2).double() * 0.5
    base.close(r.dlogp, want, 2 * ref.EPS32, 0.0, "dlogp")
    nan = gbce.preference_loss(torch.full((4,), NEG, device=DEV), [0, 2, 4], label_smoothing=eps)
    assert math.isnan(float(nan.loss))


@pytest.mark.parametrize("T", [0.5, 1.0, 2.0])
@pytest.mark.parametrize("rows,V,dtype", PLACES)
def test_teachers_of_the_lowest_value(gbce, rows, V, dtype, T):  # noqa: F811
    """A list whose logits are all at the lowest value shares its mass evenly (no rest), or leaves it to
    the rest; one among them that is not takes it."""
    g = gen(V + 12)
    x = torch.zeros((rows, V), dtype=dtype)
    x[:4] = (torch.randn((4, V), generator=g) * 2.0).to(dtype)
    idx = torch.stack([torch.randperm(V, generator=g)[:20] for _ in range(rows)])
    t = torch.zeros((rows, 20))
    t[:4] = torch.finfo(F32).min
    t[1, 3] = 1.0
    t[3, :10], idx[3, 12] = NEG, idx[3, 15]     # (a column listed twice)
    seen = t[:4].clone()
    seen[0], seen[3, 10:], seen[1][seen[1] < 0] = 0.0, 0.0, NEG
    rest = torch.zeros(rows)
    for r in (None, rest):
        low = seen.clone()
        if r is not None:
            low[[0, 2, 3]] = NEG
            r[1] = 0.5
        else:
            low[2] = 0.0
        per, dz, move = ref.distill(x[:4].float(), idx[:4], low, None if r is None else r[:4], T)
        one = torch.ones(rows, device=DEV)
        args = (gpu(x), gpu(idx), gpu(t), gpu(r))
        out = gbce.distill_fwd_bwd_fused(*args, one, T, None, "none")
        f = gbce.distill_fwd(*args, T, None, "none")
        b = gbce.distill_bwd(*args, one, f.rest_state, None, T, None, "none")
        for loss, d in ((out.loss, out.dlogits), (f.loss, b)):
            base.close(loss[:4], per, base.LOSS_TOL, ref.kl_bound(per, move))
            base.rows_close(d[:4], dz / T, dtype, floor=ref.gap_bound(move) / T)
