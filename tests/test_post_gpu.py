"""The post-training losses on the GPU against their 64-bit definitions."""

import math

import pytest
import torch

import post_ref as ref
from helpers import GRAD_FLOOR, GRAD_TOL, LOGP_TOL, LOSS_TOL

pytestmark = pytest.mark.gpu

NEG, NAN, INF = -math.inf, math.nan, math.inf
IGNORE = -100
F32, BF16 = torch.float32, torch.bfloat16
DEV = "cuda"


@pytest.fixture(scope="module")
def gbce():
    import cross_entropy_gb300 as gbce

    gbce.load_library()
    return gbce


def gen(seed):
    return torch.Generator().manual_seed(seed)


def logits_of(rows, V, dtype, g, std=2.0):
    return (torch.randn((rows, V), generator=g) * std).to(dtype)


def on_gpu(x, pad=0, shift=0):
    """x on the GPU as rows of a buffer pad columns wider, starting `shift` elements in."""
    rows, V = x.shape
    buf = torch.full((rows * (V + pad) + shift,), NAN, dtype=x.dtype, device=DEV)
    view = buf[shift:].view(rows, V + pad)[:, :V]
    view.copy_(x)
    return view


def close(got, want, tol, floor=0.0, what=""):
    got, want = got.double().cpu(), torch.as_tensor(want).double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert bool((torch.isnan(got) == torch.isnan(want)).all()), f"{what}: NaN pattern {got} {want}"
    ok = torch.isfinite(want)
    assert bool((got[~ok & ~torch.isnan(want)] == want[~ok & ~torch.isnan(want)]).all()), what
    floor = torch.as_tensor(floor).double().expand(want.shape)
    off = (got - want).abs()[ok] - tol * want.abs()[ok] - floor[ok]
    assert off.numel() == 0 or off.max() <= 0, f"{what}: {off.max():.3e} past its bound"


def rows_close(got, want, dtype, what="dlogits", floor=None):
    """Per row in norm, GRAD_TOL, the type's rounding floor and a floor of the caller's."""
    got, want = got.double().cpu(), want.double()
    assert got.shape == want.shape
    for r in range(want.shape[0]):
        if bool(torch.isnan(want[r]).any()):
            assert bool(torch.isnan(got[r]).all()), f"{what}: row {r} should be NaN"
            continue
        if not bool(want[r].any()):
            assert not bool(got[r].any()), f"{what}: row {r} should be zero"
            continue
        off = (got[r] - want[r]).norm()
        bound = GRAD_TOL[dtype] * want[r].norm() + GRAD_FLOOR[dtype] * math.sqrt(want.shape[1])
        bound += 0.0 if floor is None else float(floor[r])
        assert off <= bound, f"{what}: row {r} off by {off:.3e}, bound {bound:.3e}"


def teacher_of(x, K, g, ragged=False, rest=False, T=1.0, lead=0.0):
    rows, V = x.shape
    idx = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(rows)])
    t = x.float().gather(1, idx) + 0.7 * torch.randn((rows, K), generator=g)
    t[:, 0] += lead
    if ragged:
        keep = torch.randint(1, K + 1, (rows, 1), generator=g)
        gone = torch.arange(K) >= keep
        idx, t = idx.masked_fill(gone, -1), t.masked_fill(gone, NAN)
    r = None
    if rest:
        r = torch.logsumexp((t / T).masked_fill(idx < 0, NEG), 1) - 3.0 * torch.rand(rows, generator=g)
    return idx, t, r


def gpu(x):
    return None if x is None else x.to(DEV)


def distill_check(gbce, x, idx, t, rest, T, mask, reduction, pad=0, shift=0, status=0, seed=0):
    rows = x.shape[0]
    dtype = x.dtype
    g = torch.rand(rows if reduction == "none" else 1, generator=gen(seed + 99)) + 0.5
    per, dz, move = ref.distill(x.float(), idx, t, rest, T, mask)
    n = rows if mask is None else int((mask != 0).sum())
    up = g.double().expand(rows) / (max(n, 1) if reduction == "mean" else 1)
    want = dz * (up / T).unsqueeze(1)
    bound = ref.kl_bound(per, move).nan_to_num(0.0, 0.0, 0.0)
    floor = ref.gap_bound(move) * up / T
    xg = on_gpu(x, pad, shift)
    args = (xg, gpu(idx), gpu(t), gpu(rest))
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    fused = gbce.distill_fwd_bwd_fused(*args, gpu(g), T, gpu(mask), reduction, dev_status=flag)
    fwd = gbce.distill_fwd(*args, T, gpu(mask), reduction, dev_status=flag)
    bwd = gbce.distill_bwd(*args, gpu(g), fwd.rest_state, fwd.n_items, T, gpu(mask), reduction,
                           dev_status=flag)
    assert int(flag) == status
    for what, loss, d in (("fused", fused.loss, fused.dlogits), ("two calls", fwd.loss, bwd)):
        if reduction == "none":
            close(loss, per, LOSS_TOL, bound, what)
            assert bool((loss[torch.isfinite(loss)] >= 0).all())
        else:
            div = max(n, 1) if reduction == "mean" else 1
            close(loss, per.sum() / div, LOSS_TOL, bound.sum() / div, what)
        rows_close(d, want, dtype, what, floor)
    assert int(fused.n_items) == int(fwd.n_items) == n
    return fused


# rows, V, K, dtype, pad, shift
SHAPES = [
    (1, 1, 1, F32, 0, 0), (1, 2, 1, BF16, 0, 0), (3, 7, 7, F32, 0, 1), (2, 5, 3, BF16, 1, 3),
    (5, 64, 16, BF16, 0, 0), (64, 130, 33, F32, 3, 2), (33, 1003, 100, BF16, 5, 1),
    (300, 515, 5, BF16, 0, 0), (7, 4096, 256, F32, 0, 0), (2, 40001, 50, BF16, 7, 0),
    (5, 33000, 64, F32, 0, 0), (1, 152064, 20, BF16, 0, 0), (1, 131073, 256, F32, 0, 3),
    (160, 2048, 8, F32, 0, 0), (520, 300, 12, F32, 4, 0),
]


@pytest.mark.parametrize("rows,V,K,dtype,pad,shift", SHAPES)
@pytest.mark.parametrize("rest,ragged,T,reduction", [(False, False, 1.0, "mean"), (True, True, 0.7, "none"),
                                                     (True, False, 2.0, "sum"), (False, True, 1.0, "none")])
def test_distill(gbce, rows, V, K, dtype, pad, shift, rest, ragged, T, reduction):
    if rest and K == V:
        pytest.skip("every column is listed: a rest with mass has an infinite loss (tested below)")
    g = gen(rows * 7919 + V)
    x = logits_of(rows, V, dtype, g)
    idx, t, r = teacher_of(x, K, g, ragged, rest, T)
    mask = None
    if rows > 4:
        mask = (torch.rand(rows, generator=g) < 0.8).to(torch.uint8)
        x[mask == 0] = NAN          # what a left-out row holds is not looked at
        t[mask == 0] = NAN
        idx[mask == 0, 0] = V + 5
    distill_check(gbce, x, idx, t, r, T, mask, reduction, pad, shift, seed=V)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lead", [8.0, 17.0, 30.0, 50.0])
def test_distill_confident_rows(gbce, dtype, lead):
    """Teacher and student both led by one token, past fp32's 1 - p; then the student led by a
    column the teacher does not list."""
    g = gen(int(lead))
    x = logits_of(24, 5003, dtype, g)
    idx, t, r = teacher_of(x, 32, g, False, True, 1.0, lead + 8.0)
    r = r - lead
    x.scatter_(1, idx[:, :1], (t[:, :1] + 0.3 * torch.randn((24, 1), generator=g)).to(dtype))
    distill_check(gbce, x, idx, t, r, 1.0, None, "none")
    other = (idx.max(1, keepdim=True).values + 1) % 5003
    x.scatter_(1, other, torch.full((24, 1), lead + 12.0).to(dtype))
    distill_check(gbce, x, idx, t, None, 1.0, None, "none")


@pytest.mark.parametrize("move", [0.0, 1e-4, 1e-2])
def test_distill_of_a_student_at_its_teacher(gbce, move):
    """A loss of about move^2: no cancellation may be left of p log p - p log q."""
    g = gen(11)
    x = logits_of(16, 900, F32, g)
    idx = torch.stack([torch.randperm(900, generator=g)[:200] for _ in range(16)])
    t = x.gather(1, idx)
    away = x.double().scatter(1, idx, NEG)
    r = torch.logsumexp(away, 1).float()
    x = x + move * torch.randn(x.shape, generator=g)
    out = distill_check(gbce, x, idx, t, r, 1.0, None, "none")
    assert float(out.loss.max()) <= 4 * move * move + 1e-9


def test_distill_empty_lists_and_infinities(gbce):
    g = gen(12)
    x = logits_of(10, 600, F32, g)
    idx, t, r = teacher_of(x, 9, g, False, True)
    idx[0] = -1                       # nothing listed, a rest: q_rest = 1 = p_rest
    idx[1] = -1
    r[1] = NEG                        # nothing at all
    t[2] = NEG
    r[2] = NEG                        # entries without mass
    t[3, 2:] = NEG                    # some without
    x[4, idx[4, 3]] = NEG             # the student cannot say a listed token: an infinite loss
    t[5, 3] = NEG
    x[5, idx[5, 3]] = NEG             # ... that the teacher does not say either
    x[6, 100:] = NEG
    r[7] = NEG
    x[8] = NEG                        # one column has all the mass
    x[8, idx[8, 0]] = 3.0
    t[8, 1:] = NEG
    r[8] = NEG
    per, _, _ = ref.distill(x, idx, t, r, 1.0)
    assert per[0] == 0 and per[1] == 0 and per[2] == 0 and per[4] == INF and per[8] == 0
    distill_check(gbce, x, idx, t, r, 1.0, None, "none")
    # without a rest
    distill_check(gbce, x, idx, t, None, 1.0, None, "none")
    # every column listed and a rest with mass: the student has no mass there
    y = logits_of(3, 5, F32, g)
    iy, ty, _ = teacher_of(y, 5, g)
    ry = torch.tensor([0.0, NEG, 1.0])
    distill_check(gbce, y, iy, ty, ry, 1.0, None, "none")


def test_distill_repeats_bad_indices_and_nan(gbce):
    g = gen(13)
    x = logits_of(8, 700, BF16, g)
    idx, t, r = teacher_of(x, 12, g, False, True)
    idx[0, 5] = idx[0, 1]             # one column named twice, and one four times
    idx[1, 3] = idx[1, 7] = idx[1, 11] = idx[1, 2]
    idx[2, 4] = 700                   # outside the vocabulary
    idx[3, 0] = -7
    t[4, 6] = NAN
    t[5, 6] = INF
    r[6] = NAN
    x[7, 650] = NAN
    out = distill_check(gbce, x[:7], idx[:7], t[:7], r[:7], 1.3, None, "none", status=2)
    assert bool(torch.isnan(out.loss[2:7]).all()) and bool(torch.isfinite(out.loss[:2]).all())
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = gbce.distill_fwd_bwd_fused(gpu(x[7:]), gpu(idx[7:]), gpu(t[7:]), gpu(r[7:]), dev_status=flag)
    assert math.isnan(float(got.loss)) and bool(torch.isnan(got.dlogits).all()) and int(flag) == 0
    # a NaN at a listed column, one alone in its vector, and a whole row of them
    for where in ([int(idx[7, 0])], list(range(8, 16)), list(range(700))):
        y = logits_of(1, 700, F32, g)
        y[0, where] = NAN
        got = gbce.distill_fwd_bwd_fused(gpu(y), gpu(idx[7:]), gpu(t[7:]), gpu(r[7:]))
        assert math.isnan(float(got.loss)) and bool(torch.isnan(got.dlogits).all()), where


def test_distill_gradient_by_differences(gbce):
    g = gen(14)
    x = logits_of(2, 23, F32, g)
    idx, t, r = teacher_of(x, 6, g, False, True)
    out = gbce.distill_fwd_bwd_fused(gpu(x), gpu(idx), gpu(t), gpu(r), torch.ones(2), 0.8,
                                     reduction="none")
    for j in range(23):
        step = torch.zeros_like(x).double()
        step[:, j] = 1e-5
        hi = ref.distill(x.double() + step, idx, t, r, 0.8)[0]
        lo = ref.distill(x.double() - step, idx, t, r, 0.8)[0]
        # differences: 1e-10 of curvature, 1e-16 / 1e-5 of rounding
        close(out.dlogits[:, j], (hi - lo) / 2e-5, 2e-5, 1e-6)


@pytest.mark.parametrize("which", ["strided", "shifted", "wide"])
def test_gradients_leave_the_rest_of_their_buffer(gbce, which):
    """A dlogits of the caller's, of another stride and alignment than the logits."""
    g = gen(15)
    rows, V = 9, 1001
    x = logits_of(rows, V, BF16, g)
    idx, t, r = teacher_of(x, 10, g, False, True)
    lab = torch.randint(0, V, (rows,), generator=g)
    lab[3] = IGNORE
    adv = torch.randn(rows, generator=g)
    pad, shift = {"strided": (3, 0), "shifted": (0, 1), "wide": (64, 8)}[which]
    xg = on_gpu(x)
    for call in (lambda d: gbce.distill_fwd_bwd_fused(xg, gpu(idx), gpu(t), gpu(r), dlogits=d),
                 lambda d: gbce.policy_loss_fwd_bwd_fused(xg, gpu(lab), gpu(adv), dlogits=d),
                 lambda d: gbce.preference_loss_fwd_bwd_fused(xg, gpu(lab), [0, 2, 4, 7, 8], dlogits=d)):
        plain = call(None).dlogits
        buf = torch.full((rows * (V + pad) + shift + 32,), 7.5, dtype=BF16, device=DEV)
        view = buf[shift:shift + rows * (V + pad)].view(rows, V + pad)
        call(view[:, :V])
        assert torch.equal(view[:, :V], plain)
        assert bool((view[:, V:] == 7.5).all()) and bool((buf[:shift] == 7.5).all())
        assert bool((buf[shift + rows * (V + pad):] == 7.5).all())


# --------------------------------------------------------------------- policy

def policy_case(rows, V, dtype, g, ignored=0.2, T=1.0):
    x = logits_of(rows, V, dtype, g)
    lab = torch.randint(0, V, (rows,), generator=g)
    lead = torch.rand(rows, generator=g) * 12.0
    x.scatter_(1, lab.unsqueeze(1), (lead * T).unsqueeze(1).to(dtype))
    lp, comp, z = ref.logp_rows(x, lab, T)
    move = 0.2 * torch.randn(rows, generator=g).double()
    for edge in (math.log(0.8), math.log(1.28)):   # no row within rounding of a clip's border
        move = torch.where((move - edge).abs() < 1e-3, move + 2e-3, move)
    old = (lp - move).float()
    kl = (lp + 0.3 * torch.randn(rows, generator=g).double()).float()
    adv = torch.randn(rows, generator=g)
    if rows > 4:
        lab[torch.rand(rows, generator=g) < ignored] = IGNORE
    return x, lab, lp, comp, z, old, kl, adv


def policy_bounds(lp, adv, old, kl, loss, d, beta, dtype):
    """A log p that is off by e = LOGP_TOL |lp| moves rho by rho e and e^d by e^d e; every product and
    exp adds a few roundings, and lp - old one of its operands'."""
    e = LOGP_TOL[dtype] * lp.abs() + 4 * ref.EPS32 * (lp.abs() + 1)
    rho = torch.exp(lp - old.double()) if old is not None else torch.ones_like(lp)
    ed = torch.exp(kl.double() - lp) if beta else torch.zeros_like(lp)
    return (e * rho * adv.double().abs() + beta * e * (ed - 1).abs() + beta * e * e * ed,
            e * rho * adv.double().abs() + beta * e * ed)


@pytest.mark.parametrize("rows,V,dtype,pad,shift", [
    (1, 1, F32, 0, 0), (1, 2, BF16, 0, 0), (5, 63, F32, 0, 1), (9, 64, BF16, 3, 0), (64, 4096, F32, 0, 0),
    (33, 1003, BF16, 5, 1), (300, 515, BF16, 0, 0), (2, 40001, BF16, 7, 0), (1, 152064, BF16, 0, 0),
    (3, 131073, F32, 0, 3), (460, 2048, F32, 0, 0)])
@pytest.mark.parametrize("T,beta,reduction,has_old", [(1.0, 0.0, "mean", True), (0.7, 0.1, "none", True),
                                                      (1.3, 0.05, "sum", False)])
def test_policy(gbce, rows, V, dtype, pad, shift, T, beta, reduction, has_old):
    g = gen(rows * 31 + V)
    x, lab, lp, comp, z, old, kl, adv = policy_case(rows, V, dtype, g, T=T)
    old = old if has_old else None
    live = lab >= 0
    loss, d = ref.policy(lp, adv.double(), None if old is None else old.double(), kl.double(), 0.2, 0.28,
                         beta)
    lb, db = policy_bounds(lp, adv, old, kl, loss, d, beta, dtype)
    gr = torch.rand(rows if reduction == "none" else 1, generator=g) + 0.5
    n = int(live.sum())
    up = gr.double().expand(rows) / (n if reduction == "mean" else 1) * live
    xg = on_gpu(x.masked_fill(~live.unsqueeze(1), NAN), pad, shift)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    opt = dict(clip_low=0.2, clip_high=0.28, kl_beta=beta, reduction=reduction)
    out = gbce.policy_loss_fwd_bwd_fused(xg, gpu(lab), gpu(adv), gpu(old), gpu(kl) if beta else None, gpu(gr),
                                         temperature=T, dev_status=flag, **opt)
    assert int(flag) == 0 and int(out.n_items) == n
    close(out.logp, torch.where(live, lp, 0.0 * lp), LOGP_TOL[dtype], 2.0 ** -148, "logp")
    zero = torch.zeros_like(loss)
    loss, lb = torch.where(live, loss, zero), torch.where(live, lb, zero)
    if reduction == "none":
        close(out.loss, loss, LOSS_TOL, lb, "loss")
    else:
        div = n if reduction == "mean" else 1
        close(out.loss, loss.sum() / div, 0.0, ((LOSS_TOL * loss.abs() + lb) / div).sum(), "loss")
    want = ref.softmax_grad(z, lab.clamp(min=0), comp, -d * up, T)
    got = out.dlogits.double().cpu()
    for r in range(rows):
        if not live[r]:
            assert not bool(got[r].any())
            continue
        unit = ref.softmax_grad(z[r:r + 1], lab[r:r + 1], comp[r:r + 1], torch.ones(1).double(), T).norm()
        bound = GRAD_TOL[dtype] * want[r].norm() + up[r] * db[r] * unit + GRAD_FLOOR[dtype] * math.sqrt(V)
        assert (got[r] - want[r]).norm() <= bound, r
    # the same from log-probs
    mask = live.to(torch.uint8)
    rows_out = gbce.policy_loss(gpu(lp.float().masked_fill(~live, NAN)), gpu(adv), gpu(old),
                                gpu(kl) if beta else None, gpu(gr), gpu(mask), **opt)
    assert int(rows_out.n_items) == n
    close(rows_out.dlogp, torch.where(live, d * up, zero), LOSS_TOL, up * db, "dlogp")
    if reduction == "none":
        close(rows_out.loss, loss, LOSS_TOL, lb, "loss of log-probs")


def test_policy_clip_sides_and_borders(gbce):
    """Both signs of A on each side of both clips; at a border itself the unclipped gradient."""
    lp = torch.full((8,), -2.0)
    old = lp - torch.tensor([0.5, 0.5, -0.5, -0.5, 0.0, 0.0, 100.0, -100.0])
    adv = torch.tensor([1.0, -1.0, 1.0, -1.0, 1.0, -1.0, 0.0, 2.0])
    out = gbce.policy_loss(gpu(lp), gpu(adv), gpu(old), None, torch.ones(8), clip_low=0.0, clip_high=0.0,
                           reduction="none")
    e = math.exp(0.5)
    close(out.loss, torch.tensor([-1.0, e, -1 / e, 1.0, -1.0, 1.0, 0.0, 0.0]).double(), 1e-6, 1e-30)
    close(out.dlogp, torch.tensor([0.0, e, -1 / e, 0.0, -1.0, 1.0, 0.0, 0.0]).double(), 1e-6, 1e-30)
    # no clip above, an infinite ratio: clipped below for A > 0, infinite for A < 0
    big = gbce.policy_loss(gpu(torch.zeros(3)), gpu(torch.tensor([1.0, -1.0, 0.0])), gpu(torch.full((3,), -200.0)),
                           None, torch.ones(3), clip_high=0.2, reduction="none")
    close(big.loss, torch.tensor([-1.2, INF, 0.0]).double(), 1e-6)
    free = gbce.policy_loss(gpu(lp), gpu(adv.abs()), gpu(old), None, torch.ones(8), clip_high=INF,
                            reduction="none")
    close(free.loss[:1], torch.tensor([-e]).double(), 1e-6)


def test_policy_everything_left_out_bad_labels_and_nan(gbce):
    g = gen(21)
    x = gpu(logits_of(6, 300, F32, g))
    lab = torch.full((6,), IGNORE)
    adv = gpu(torch.ones(6))
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = gbce.policy_loss_fwd_bwd_fused(x, gpu(lab), adv, dev_status=flag)
    assert float(out.loss) == 0 and not bool(out.dlogits.any()) and int(out.n_items) == 0
    none = gbce.policy_loss(adv, adv, row_mask=gpu(torch.zeros(6)))
    assert float(none.loss) == 0 and not bool(none.dlogp.any()) and int(none.n_items) == 0
    lab = torch.tensor([3, 300, 5, -7, 8, 9])
    x[4, 200] = NAN
    x[5] = NAN
    out = gbce.policy_loss_fwd_bwd_fused(x, gpu(lab), adv, None, None, torch.ones(6), reduction="none",
                                         dev_status=flag)
    assert int(flag) == 1
    bad = torch.tensor([False, True, False, True, True, True])
    assert torch.equal(torch.isnan(out.loss).cpu(), bad) and torch.equal(torch.isnan(out.logp).cpu(), bad)
    assert torch.equal(torch.isnan(out.dlogits).all(1).cpu(), bad)
    assert bool(torch.isfinite(out.dlogits[[0, 2]]).all())


def test_policy_takes_a_value_per_sequence(gbce):
    g = gen(22)
    x = gpu(logits_of(24, 200, F32, g)).view(4, 6, 200)
    lab = gpu(torch.randint(0, 200, (4, 6), generator=g))
    adv = gpu(torch.randn((4, 1), generator=g))
    a = gbce.policy_loss_fwd_bwd_fused(x, lab, adv)
    b = gbce.policy_loss_fwd_bwd_fused(x.view(24, 200), lab.view(24), adv.expand(4, 6).reshape(24))
    assert a.dlogits.shape == x.shape and torch.equal(a.dlogits.view(24, 200), b.dlogits)
    assert torch.equal(a.loss, b.loss)
    with pytest.raises(ValueError):
        gbce.policy_loss_fwd_bwd_fused(x, lab, adv[:3])
    with pytest.raises(gbce.GbceError):
        gbce.policy_loss_fwd_bwd_fused(x, lab, adv, kl_beta=0.1)


# ----------------------------------------------------------------- preference

def offsets_of(rows, pairs, g, outside=0):
    cuts = torch.sort(torch.randint(0, rows - outside + 1, (2 * pairs - 1,), generator=g)).values
    return torch.cat([torch.tensor([min(outside, 1)]), cuts.clamp(min=min(outside, 1)),
                      torch.tensor([rows - outside])])


@pytest.mark.parametrize("rows,V,pairs,dtype,pad,outside", [
    (2, 5, 1, F32, 0, 0), (1, 30, 1, BF16, 0, 0), (3, 64, 5, F32, 0, 0), (40, 1003, 3, BF16, 5, 2),
    (64, 4096, 2, F32, 0, 0), (700, 260, 40, BF16, 0, 3), (12, 40001, 2, BF16, 0, 1), (900, 64, 2, F32, 3, 0)])
@pytest.mark.parametrize("kind,average,has_ref,reduction,beta,eps,margin", [
    ("sigmoid", False, True, "mean", 0.1, 0.0, 0.0), ("sigmoid", True, False, "sum", 2.0, 0.1, 0.5),
    ("squared", True, True, "none", 0.3, 0.0, 0.0)])
def test_preference(gbce, rows, V, pairs, dtype, pad, outside, kind, average, has_ref, reduction, beta, eps,
                    margin):
    g = gen(rows * 17 + V)
    T = 0.9
    x, lab, lp, comp, z, _, kl, _ = policy_case(rows, V, dtype, g, T=T)
    off = offsets_of(rows, pairs, g, outside)
    live = lab >= 0
    inside = (torch.arange(rows) >= off[0]) & (torch.arange(rows) < off[-1])
    r = kl.double() if has_ref else None
    loss, score, drow, pair = ref.preference(lp, off, r, live, beta, margin, eps, kind, average)
    gr = torch.rand(pairs if reduction == "none" else 1, generator=g) + 0.5
    up = gr.double().expand(pairs) / (pairs if reduction == "mean" else 1)
    uprow = torch.where(pair >= 0, up[pair.clamp(min=0)], torch.zeros(rows).double())
    # a log p within LOGP_TOL: the scores move by the sum of that over their rows, the loss by its
    # slope times it (beta at most, 2 |e| and 1 for the squared one), and the slope by its own
    e_row = (LOGP_TOL[dtype] * lp.abs() + 2 * ref.EPS32 * (kl.double().abs() if has_ref else 0.0)) * (live & inside)
    e_pair = torch.zeros(pairs).double().index_add_(0, pair.clamp(min=0), e_row)
    h = score[:pairs] - score[pairs:]
    if kind == "squared":
        eh = 2 * (h - 0.5 / beta).abs() * e_pair + e_pair ** 2
        es = 2 * e_pair
    else:
        eh, es = beta * e_pair, beta * beta * e_pair
    seen = inside & live
    xg = on_gpu(x.masked_fill(~seen.unsqueeze(1), NAN), pad)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    opt = dict(beta=beta, margin=margin, label_smoothing=eps, kind=kind, average=average, reduction=reduction,
               dev_status=flag)
    out = gbce.preference_loss_fwd_bwd_fused(xg, gpu(lab), gpu(off), gpu(kl) if has_ref else None, gpu(gr),
                                             temperature=T, **opt)
    close(out.logp, torch.where(seen, lp, 0.0 * lp), LOGP_TOL[dtype], 2.0 ** -148, "logp")
    e_seq = torch.zeros(2 * pairs).double()
    for s in range(2 * pairs):
        e_seq[s] = e_row[int(off[s]):int(off[s + 1])].sum()
    close(out.seq_score, score, 2 * ref.EPS32, e_seq, "score")
    bound = LOSS_TOL * loss.abs() + eh
    if reduction == "none":
        close(out.loss, loss, 0.0, bound, "loss")
    else:
        div = pairs if reduction == "mean" else 1
        close(out.loss, loss.sum() / div, 0.0, bound.sum() / div, "loss")
    want = ref.softmax_grad(z, lab.clamp(min=0), comp, -drow * uprow, T)
    got = out.dlogits.double().cpu()
    for i in range(rows):
        if not seen[i]:
            assert not bool(got[i].any()), i
            continue
        unit = ref.softmax_grad(z[i:i + 1], lab[i:i + 1], comp[i:i + 1], torch.ones(1).double(), T).norm()
        b = GRAD_TOL[dtype] * want[i].norm() + uprow[i] * es[pair[i]] * unit + GRAD_FLOOR[dtype] * math.sqrt(V)
        assert (got[i] - want[i]).norm() <= b, i
    # from log-probs, rows left out holding anything
    mask = live.to(torch.uint8)
    lpg = gpu(lp.float().masked_fill(~seen, NAN))
    two = gbce.preference_loss(lpg, gpu(off), gpu(kl) if has_ref else None, gpu(gr), gpu(mask), **opt)
    assert int(flag) == 0
    close(two.seq_score, score, 2 * ref.EPS32, e_seq, "score of log-probs")
    close(two.dlogp, torch.where(seen, drow * uprow, 0.0 * drow), LOSS_TOL,
          uprow * torch.where(pair >= 0, es[pair.clamp(min=0)], torch.zeros(rows).double()), "dlogp")


def test_preference_bad_offsets_stay_inside(gbce):
    g = gen(31)
    x = gpu(logits_of(12, 90, F32, g))
    lab = gpu(torch.randint(0, 90, (12,), generator=g))
    good = gbce.preference_loss_fwd_bwd_fused(x, lab, [0, 3, 6, 9, 12], reduction="none", grad_out=torch.ones(2))
    for off, bad in (([0, 3, 6, 9, 13], [0, 1]), ([-1, 3, 6, 9, 12], [0, 1]), ([0, 6, 3, 9, 12], [0, 1]),
                     ([0, 3, 6, 5, 12], [0, 1]), ([0, 3, 1 << 40, 9, 12], [0, 1])):
        flag = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = gbce.preference_loss_fwd_bwd_fused(x, lab, off, reduction="none", grad_out=torch.ones(2),
                                                 dev_status=flag)
        two = gbce.preference_loss(good.logp, off, reduction="none", grad_out=torch.ones(2))
        assert int(flag) == 2
        for loss in (out.loss, two.loss):
            assert bool(torch.isnan(loss).any())
    # no rows at all: both scores 0
    none = gbce.preference_loss(torch.empty(0, device=DEV), [0, 0, 0])
    assert abs(float(none.loss) - math.log(2.0)) < 1e-7 and not bool(none.seq_score.any())
    empty = gbce.preference_loss_fwd_bwd_fused(torch.empty((0, 9), device=DEV), torch.empty(0), [0, 0, 0])
    assert abs(float(empty.loss) - math.log(2.0)) < 1e-7 and empty.dlogits.shape == (0, 9)


def test_preference_of_a_batch(gbce):
    g = gen(32)
    x = gpu(logits_of(24, 70, F32, g)).view(4, 6, 70)
    lab = gpu(torch.randint(0, 70, (4, 6), generator=g))
    a = gbce.preference_loss_fwd_bwd_fused(x, lab)
    b = gbce.preference_loss_fwd_bwd_fused(x.view(24, 70), lab.view(24), [0, 6, 12, 18, 24])
    assert torch.equal(a.dlogits.view(24, 70), b.dlogits) and torch.equal(a.loss, b.loss)
    with pytest.raises(ValueError):
        gbce.preference_loss_fwd_bwd_fused(x[:3], lab[:3])
    with pytest.raises(ValueError):
        gbce.preference_loss_fwd_bwd_fused(x, lab, [0, 12, 18, 24])


# ------------------------------------------------------------- as they are used

def test_empty_calls(gbce):
    x, i = torch.empty((0, 9), device=DEV), torch.empty((0, 3), dtype=torch.int64, device=DEV)
    t = torch.empty((0, 3), device=DEV)
    out = gbce.distill_fwd_bwd_fused(x, i, t)
    assert float(out.loss) == 0 and int(out.n_items) == 0 and out.dlogits.shape == (0, 9)
    f = gbce.distill_fwd(x, i, t)
    assert float(f.loss) == 0
    gbce.distill_bwd(x, i, t, None, torch.ones(1), f.rest_state, f.n_items)
    p = gbce.policy_loss_fwd_bwd_fused(x, i[:, 0], t[:, 0])
    assert float(p.loss) == 0 and int(p.n_items) == 0
    q = gbce.policy_loss(t[:, 0], t[:, 0])
    assert float(q.loss) == 0 and int(q.n_items) == 0


def test_losses_of_a_linear_head(gbce):
    """Log-probs of a head that keeps no logits, the loss from them, and its gradient: as the loss of
    the logits and their product."""
    g = gen(41)
    h = gpu(torch.randn((40, 48), generator=g))
    w = gpu(torch.randn((1001, 48), generator=g) * 0.4)
    lab = torch.randint(0, 1001, (40,), generator=g)
    mask = (torch.rand(40, generator=g) < 0.8).to(torch.uint8)
    adv = gpu(torch.randn(40, generator=g))
    kept = gpu(lab.masked_fill(mask == 0, IGNORE))
    x = h.double() @ w.double().t()
    lp, _, _ = ref.logp_rows(x.cpu(), lab, 1.0)
    old = gpu((lp + 0.1 * torch.randn(40, generator=g)).float())
    kl = gpu((lp + 0.1 * torch.randn(40, generator=g)).float())
    logp, state = gbce.linear_selective_logsoftmax(h, w, gpu(lab), 1.0, gpu(mask), with_state=True)
    for name in ("policy", "preference"):
        if name == "policy":
            a = gbce.policy_loss(logp, adv, old, kl, None, gpu(mask), kl_beta=0.1)
            b = gbce.policy_loss_fwd_bwd_fused(x.float(), kept, adv, old, kl, kl_beta=0.1)
        else:
            off = [0, 9, 20, 31, 40]
            a = gbce.preference_loss(logp, off, kl, None, gpu(mask))
            b = gbce.preference_loss_fwd_bwd_fused(x.float(), kept, off, kl)
        dh, dw = gbce.linear_selective_logsoftmax_bwd(h, w, gpu(lab), a.dlogp, logp, state, 1.0, gpu(mask))
        assert abs(float(a.loss) - float(b.loss)) <= 2e-5 * abs(float(b.loss)) + 1e-6
        dx = b.dlogits.double()
        for got, want in ((dh, dx @ w.double()), (dw, dx.t() @ h.double())):
            assert (got.double() - want).norm() <= 1e-4 * want.norm(), name


def test_a_captured_step_follows_its_inputs(gbce):
    """A step of all three losses, captured and replayed on new inputs; an eager call in between."""
    g = gen(42)
    rows, V, K = 21, 1003, 9

    def inputs(seed):
        q = gen(seed)
        x = logits_of(rows, V, BF16, q)
        idx, t, r = teacher_of(x, K, q, False, True)
        lab = torch.randint(0, V, (rows,), generator=q)
        return [gpu(v) for v in (x, idx, t, r, lab, torch.randn(rows, generator=q))]

    def step(x, idx, t, r, lab, adv, off):
        a = gbce.distill_fwd_bwd_fused(x, idx, t, r, one)
        f = gbce.distill_fwd(x, idx, t, r)
        b = gbce.distill_bwd(x, idx, t, r, one, f.rest_state, f.n_items)
        p = gbce.policy_loss_fwd_bwd_fused(x, lab, adv, None, None, one)
        d = gbce.preference_loss_fwd_bwd_fused(x, lab, off, None, one)
        e = gbce.policy_loss(p.logp, adv, None, None, one)
        u = gbce.preference_loss(d.logp, off, None, one)
        return [a.loss, a.dlogits, f.loss, b, p.loss, p.dlogits, d.loss, d.dlogits, d.seq_score, e.dlogp, u.dlogp]

    one = torch.ones(1, device=DEV)
    off = torch.tensor([0, 5, 9, 9, 20], device=DEV)
    held = inputs(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*held, off)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*held, off)
    for seed in (2, 3):
        new = inputs(seed)
        for a, b in zip(held, new):
            a.copy_(b)
        graph.replay()
        eager = step(*new, off)
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert torch.equal(a, b)


def test_another_stream(gbce):
    """Calls on a given stream, one after another with their inputs made there."""
    g = gen(43)
    s = torch.cuda.Stream()
    x = gpu(logits_of(200, 5000, BF16, g))
    idx, t, r = teacher_of(x.cpu(), 7, g, False, True)
    lab = gpu(torch.randint(0, 5000, (200,), generator=g))
    adv = gpu(torch.randn(200, generator=g))
    idx, t, r = gpu(idx), gpu(t), gpu(r)
    want = gbce.distill_fwd_bwd_fused(x, idx, t, r), gbce.policy_loss_fwd_bwd_fused(x, lab, adv)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        y = x.clone()
    a = gbce.distill_fwd_bwd_fused(y, idx, t, r, stream=s)
    b = gbce.policy_loss_fwd_bwd_fused(y, lab, adv, stream=s)
    s.synchronize()
    for u, v in zip((a, b), want):
        assert torch.equal(u.loss, v.loss) and torch.equal(u.dlogits, v.dlogits)


def test_rows_past_32_bits(gbce):
    """The last rows of a matrix of more than 2^32 bytes and 2^31 elements."""
    rows, V = 14200, 152064
    x = torch.zeros((rows, V), dtype=BF16, device=DEV)
    g = gen(44)
    tail = logits_of(3, V, BF16, g)
    x[-3:] = gpu(tail)
    idx = torch.full((rows, 2), -1)
    idx[-3:] = torch.randint(0, V, (3, 2), generator=g)
    idx[-3:, 1] = (idx[-3:, 0] + 77) % V
    t = torch.zeros((rows, 2))
    mask = torch.zeros(rows, dtype=torch.uint8)
    mask[-3:] = 1
    out = gbce.distill_fwd_bwd_fused(x, gpu(idx), gpu(t), None, None, 1.0, gpu(mask))
    per, dz, move = ref.distill(tail.float(), idx[-3:], t[-3:], None, 1.0)
    close(out.loss, per.mean(), LOSS_TOL, ref.kl_bound(per, move).mean())
    rows_close(out.dlogits[-3:], dz / 3.0, BF16)
    assert not bool(out.dlogits[:-3].any())


@pytest.mark.parametrize("rows,V,dtype,pad", [(3, 40001, BF16, 7), (30, 70001, BF16, 3), (5, 33001, F32, 1)])
def test_split_rows_of_another_phase(gbce, rows, V, dtype, pad):
    """Few long rows (each one's slices on several CTAs) whose gradient lies at another offset modulo
    16 bytes, the listed columns on both sides of every slice's ends."""
    g = gen(V)
    x = logits_of(rows, V, dtype, g)
    K = 256
    ends = torch.cat([torch.arange(16), torch.arange(V - 16, V),
                      *[V * i // 8 + torch.arange(-12, 12) for i in range(1, 8)]])
    more = torch.randperm(V - 100, generator=g) + 50
    cols = torch.unique(torch.cat([ends, more[:400]]))
    idx = torch.stack([cols[torch.randperm(cols.numel(), generator=g)[:K]] for _ in range(rows)])
    t = x.float().gather(1, idx) + torch.randn((rows, K), generator=g)
    r = torch.logsumexp(t, 1) - 1.0
    distill_check(gbce, x, idx, t, r, 1.0, None, "none", pad=pad)
    lab = cols[torch.randint(0, cols.numel(), (rows,), generator=g)]
    xg = on_gpu(x, pad)
    lp, comp, z = ref.logp_rows(x, lab, 1.0)
    out = gbce.policy_loss_fwd_bwd_fused(xg, gpu(lab), gpu(torch.ones(rows)), None, None, torch.ones(rows),
                                         reduction="none")
    rows_close(out.dlogits, ref.softmax_grad(z, lab, comp, torch.ones(rows).double(), 1.0), dtype)
    pref = gbce.preference_loss_fwd_bwd_fused(xg, gpu(lab), [0, 1, rows], beta=1.0, average=True)
    _, _, d, _ = ref.preference(lp, [0, 1, rows], None, lab >= 0, 1.0, 0.0, 0.0, "sigmoid", True)
    e = 2 * LOGP_TOL[dtype] * float(lp.abs().max())     # of each score's mean, times the slope's slope <= 1
    unit = ref.softmax_grad(z, lab, comp, torch.ones(rows).double(), 1.0).norm(dim=1)
    rows_close(pref.dlogits, ref.softmax_grad(z, lab, comp, -d, 1.0), dtype, floor=e * unit)


@pytest.mark.parametrize("rows", [131072, 131073, 300001])
@pytest.mark.parametrize("masked", [False, True])
def test_long_vectors_of_log_probs(gbce, rows, masked):
    """On both sides of where the policy loss of log-probs takes a grid instead of one cluster."""
    g = gen(rows)
    lp = -3.0 * torch.rand(rows, generator=g)
    adv = torch.randn(rows, generator=g)
    old = lp - 0.05 * torch.randn(rows, generator=g)
    mask = (torch.rand(rows, generator=g) < 0.3).to(torch.uint8) if masked else None
    live = torch.ones(rows, dtype=torch.bool) if mask is None else mask != 0
    loss, d = ref.policy(lp.double(), adv.double(), old.double(), None, 0.9, 5.0, 0.0)
    n = int(live.sum())
    for reduction, div in (("mean", n), ("sum", 1)):
        out = gbce.policy_loss(gpu(lp), gpu(adv), gpu(old), None, torch.full((1,), 2.0), gpu(mask), clip_low=0.9,
                               clip_high=5.0, reduction=reduction)
        assert int(out.n_items) == n
        kept = loss * live
        # an exp and two products a row (four roundings), 48-bit sums, one rounding of the result
        close(out.loss, kept.sum() / div, 2 * ref.EPS32, 6 * ref.EPS32 * kept.abs().sum() / div)
        close(out.dlogp, 2.0 * d * live / div, 8 * ref.EPS32)
    per = gbce.policy_loss(gpu(lp), gpu(adv), gpu(old), None, None, gpu(mask), clip_low=0.9, clip_high=5.0,
                           reduction="none", want_grad=False)
    assert per.dlogp is None
    close(per.loss, loss * live, 6 * ref.EPS32)


def test_same_bits_again_and_beside_another_call(gbce):
    """The same call gives the same bits, also while another runs on another stream, and rows that
    come in several waves of CTAs give what they give alone."""
    g = gen(51)
    rows, V, K = 2000, 2048, 20
    x = gpu(logits_of(rows, V, BF16, g))
    idx, t, r = (gpu(v) for v in teacher_of(x.cpu(), K, g, False, True))
    lab = gpu(torch.randint(0, V, (rows,), generator=g))
    adv = gpu(torch.randn(rows, generator=g))
    off = torch.tensor([0, 300, 900, 1500, 2000], device=DEV)

    def calls():
        a = gbce.distill_fwd_bwd_fused(x, idx, t, r)
        b = gbce.policy_loss_fwd_bwd_fused(x, lab, adv)
        c = gbce.preference_loss_fwd_bwd_fused(x, lab, off)
        return [a.loss, a.dlogits, b.loss, b.dlogits, c.loss, c.dlogits, c.seq_score]

    first = calls()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for s in (s1, s2):
            with torch.cuda.stream(s):
                outs.append(calls())
    torch.cuda.synchronize()
    for out in outs:
        for a, b in zip(first, out):
            assert torch.equal(a, b)
    one = gbce.distill_fwd_bwd_fused(x[7:9], idx[7:9], t[7:9], r[7:9], torch.full((1,), 2.0 / rows))
    # (rows of another wave, shape or split: the same formula, other orders of the same sums)
    rows_close(one.dlogits, first[1][7:9].double().cpu(), BF16)


@pytest.mark.parametrize("rows,V", [(300, 152064), (800, 40000), (470, 100003)])
def test_long_rows_in_every_shape(gbce, rows, V):
    """Several rows per CTA of the larger shapes, one row in three left out."""
    g = gen(V)
    x = torch.randn((rows, V), device=DEV).mul_(2.0).to(BF16)
    idx = torch.randint(0, V // 8, (rows, 8), generator=g) + torch.arange(8) * (V // 8)
    lab = torch.randint(0, V, (rows,), generator=g)
    t = torch.randn((rows, 8), generator=g) + 8.0
    mask = (torch.arange(rows) % 3 != 1).to(torch.uint8)
    kept = lab.masked_fill(mask == 0, IGNORE)
    some = [0, 1, 2, rows // 2, rows - 2, rows - 1]
    out = gbce.distill_fwd_bwd_fused(x, gpu(idx), gpu(t), None, torch.ones(rows), 1.0, gpu(mask), "none")
    f = gbce.distill_fwd(x, gpu(idx), gpu(t), None, 1.0, gpu(mask), "none")
    b = gbce.distill_bwd(x, gpu(idx), gpu(t), None, torch.ones(rows), f.rest_state, None, 1.0, gpu(mask), "none")
    per, dz, move = ref.distill(x[some].cpu().float(), idx[some], t[some], None, 1.0, mask[some])
    for loss, d in ((out.loss, out.dlogits), (f.loss, b)):
        close(loss[some], per, LOSS_TOL, ref.kl_bound(per, move))
        rows_close(d[some], dz, BF16, floor=ref.gap_bound(move))
        assert not bool(d[1::3].any()) and not bool(loss[1::3].any())
    assert bool((out.dlogits.sum(1).abs() < 0.05).all())
    p = gbce.policy_loss_fwd_bwd_fused(x, gpu(kept), gpu(torch.ones(rows)), None, None, torch.ones(rows),
                                       reduction="none")
    lp, comp, z = ref.logp_rows(x[some].cpu(), lab[some], 1.0)
    live = mask[some].bool()
    close(p.logp[some], torch.where(live, lp, 0 * lp), LOGP_TOL[BF16])
    rows_close(p.dlogits[some], ref.softmax_grad(z, lab[some], comp, live.double(), 1.0), BF16)
    q = gbce.preference_loss_fwd_bwd_fused(x, gpu(kept), [0, rows // 2, rows], average=True, beta=1.0)
    close(q.logp[some], torch.where(live, lp, 0 * lp), LOGP_TOL[BF16])
    slope = float(q.dlogits[0].float().norm()) / float(p.dlogits[0].float().norm())
    half = int((mask[:rows // 2] != 0).sum())
    h = q.seq_score.double().cpu()
    want = float(torch.sigmoid(h[1] - h[0])) / half
    assert abs(slope - want) <= 8e-3 * want      # two bf16 gradients' norms


@pytest.mark.parametrize("V,dtype", [(64, BF16), (600, F32), (5000, BF16)])
def test_rows_left_out_between_others_change_nothing(gbce, V, dtype):
    """A kept row has the same bits whatever rows lie between: short rows, of which a CTA takes
    several, with every pattern of rows left out."""
    g = gen(V + 1)
    rows, K = 6000, 6
    x = gpu(logits_of(rows, V, dtype, g))
    idx, t, r = (gpu(v) for v in teacher_of(x.cpu(), K, g, False, True))
    lab = gpu(torch.randint(0, V, (rows,), generator=g))
    adv = gpu(torch.randn(rows, generator=g))
    one = torch.ones(rows, device=DEV)
    a = gbce.distill_fwd_bwd_fused(x, idx, t, r, one, 1.0, None, "none")
    f = gbce.distill_fwd(x, idx, t, r, 1.0, None, "none")
    b = gbce.policy_loss_fwd_bwd_fused(x, lab, adv, None, None, one, reduction="none")
    n = torch.arange(rows, device=DEV)
    for keep in (n % 2 == 0, n % 3 == 1, (n // 3) % 2 == 0, torch.rand(rows, generator=g).to(DEV) < 0.5):
        for _ in range(3):
            c = gbce.distill_fwd_bwd_fused(x, idx, t, r, one, 1.0, keep, "none")
            h = gbce.distill_fwd(x, idx, t, r, 1.0, keep, "none")
            d = gbce.policy_loss_fwd_bwd_fused(x, lab.masked_fill(~keep, IGNORE), adv, None, None, one,
                                               reduction="none")
            for got, want in ((c.loss, a.loss), (c.dlogits, a.dlogits), (h.loss, f.loss),
                              (h.rest_state, f.rest_state), (d.loss, b.loss), (d.dlogits, b.dlogits)):
                assert torch.equal(got[keep], want[keep])
            assert not bool(c.dlogits[~keep].any()) and not bool(d.dlogits[~keep].any())
