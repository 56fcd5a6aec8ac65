"""Host-side checks of the post-training losses: every refusal returns before
any CUDA call, so none of this needs a GPU."""

import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from cross_entropy_gb300 import build

    path = build.build()
    import cross_entropy_gb300 as gbce

    return gbce.load_library(path)


def far(i):
    """Addresses that do not overlap for these sizes; never dereferenced."""
    return 0x100000 + i * (1 << 24)


BIG = 1 << 40
NAN, INF = float("nan"), float("inf")


def policy_options(**kw):
    from cross_entropy_gb300.losses import PolicyOptions

    a = dict(clip_low=0.2, clip_high=0.2, kl_beta=0.1)
    a.update(kw)
    return PolicyOptions(**a)


def preference_options(**kw):
    from cross_entropy_gb300.losses import PreferenceOptions

    a = dict(beta=0.1, margin=0.0, label_smoothing=0.0, kind=0, average=0)
    a.update(kw)
    return PreferenceOptions(**a)


def distill_fwd(lib, **kw):
    a = dict(x=far(0), dt=1, rows=4, vocab=100, xs=100, idx=far(1), k=8, t=far(2), rest=None, T=1.0,
             mask=None, red=2, loss=far(3), state=far(4), n=far(5), wk=far(6), wb=BIG, st=None, s=None)
    a.update(kw)
    return lib.distill_fwd(*a.values())


def distill_bwd(lib, **kw):
    a = dict(x=far(0), dt=1, rows=4, vocab=100, xs=100, idx=far(1), k=8, t=far(2), rest=None, T=1.0,
             mask=None, red=2, g=far(3), state=far(4), n=far(5), d=far(7), ds=100, st=None, s=None)
    a.update(kw)
    return lib.distill_bwd(*a.values())


def distill_fused(lib, **kw):
    a = dict(x=far(0), dt=1, rows=4, vocab=100, xs=100, idx=far(1), k=8, t=far(2), rest=None, T=1.0,
             mask=None, red=2, g=far(3), loss=far(4), n=far(5), d=far(7), ds=100, wk=far(6), wb=BIG,
             st=None, s=None)
    a.update(kw)
    return lib.distill_fwd_bwd_fused(*a.values())


def policy_fused(lib, opt=None, **kw):
    opt = policy_options() if opt is None else opt
    a = dict(x=far(0), dt=1, rows=4, vocab=100, xs=100, lab=far(1), ign=-100, T=1.0, adv=far(2),
             old=far(3), ref=far(4), options=ctypes.addressof(opt), red=2, g=far(5), loss=far(8), lp=None,
             n=None, d=far(7), ds=100, wk=far(6), wb=BIG, st=None, s=None)
    a.update(kw)
    return lib.policy_loss_fwd_bwd_fused(*a.values())


def policy(lib, opt=None, **kw):
    opt = policy_options() if opt is None else opt
    a = dict(lp=far(0), rows=4, mask=None, adv=far(2), old=far(3), ref=far(4),
             options=ctypes.addressof(opt), red=2, g=far(5), loss=far(8), d=far(7), n=None, wk=far(6),
             wb=BIG, s=None)
    a.update(kw)
    return lib.policy_loss(*a.values())


def preference_fused(lib, opt=None, **kw):
    opt = preference_options() if opt is None else opt
    a = dict(x=far(0), dt=1, rows=4, vocab=100, xs=100, lab=far(1), ign=-100, T=1.0, off=far(2),
             pairs=2, ref=None, options=ctypes.addressof(opt), red=2, g=far(5), loss=far(8), lp=None,
             score=None, d=far(7), ds=100, wk=far(6), wb=BIG, st=None, s=None)
    a.update(kw)
    return lib.preference_loss_fwd_bwd_fused(*a.values())


def preference(lib, opt=None, **kw):
    opt = preference_options() if opt is None else opt
    a = dict(lp=far(0), rows=4, mask=None, off=far(2), pairs=2, ref=None, options=ctypes.addressof(opt),
             red=2, g=far(5), loss=far(8), d=far(7), score=None, wk=far(6), wb=BIG, st=None, s=None)
    a.update(kw)
    return lib.preference_loss(*a.values())


LOGITS = [(dict(dt=7), 2), (dict(x=far(0) + 1), 2), (dict(x=None), 1), (dict(vocab=0), 1),
          (dict(vocab=1 << 31), 1), (dict(xs=99), 1), (dict(rows=-1), 1), (dict(rows=1 << 30), 1),
          (dict(xs=1 << 61), 1), (dict(T=0.0), 1), (dict(T=NAN), 1), (dict(T=INF), 1), (dict(T=-1.0), 1),
          (dict(red=3), 1), (dict(red=-1), 1)]
SPACE = [(dict(wk=None), 4), (dict(wk=far(6) + 8), 4), (dict(wb=64), 4), (dict(loss=None), 1)]
DLOGITS = [(dict(d=None), 1), (dict(ds=99), 1), (dict(d=far(7) + 1), 2), (dict(d=far(0)), 1),
           (dict(d=far(0) + 600), 1), (dict(ds=1 << 61), 1), (dict(g=None), 1)]
LISTS = [(dict(idx=None), 1), (dict(t=None), 1), (dict(k=0), 1), (dict(k=257), 1)]
OPTIONS = [dict(clip_low=-0.1), dict(clip_low=1.1), dict(clip_low=NAN), dict(clip_high=-0.1),
           dict(clip_high=NAN), dict(kl_beta=-0.1), dict(kl_beta=NAN), dict(kl_beta=INF)]
PAIRED = [dict(beta=0.0), dict(beta=-1.0), dict(beta=NAN), dict(beta=INF), dict(margin=NAN),
          dict(margin=INF), dict(label_smoothing=-0.1), dict(label_smoothing=0.5),
          dict(label_smoothing=NAN), dict(kind=2), dict(kind=-1), dict(kind=1, margin=0.5),
          dict(kind=1, label_smoothing=0.1)]


@pytest.mark.parametrize("kw,code", LOGITS + SPACE + LISTS)
def test_distill_fwd_refusals(lib, kw, code):
    assert distill_fwd(lib, **kw) == code


@pytest.mark.parametrize("kw,code", LOGITS + DLOGITS + LISTS + [(dict(state=None), 1), (dict(n=None), 1)])
def test_distill_bwd_refusals(lib, kw, code):
    assert distill_bwd(lib, **kw) == code


@pytest.mark.parametrize("kw,code", LOGITS + SPACE + DLOGITS + LISTS)
def test_distill_fused_refusals(lib, kw, code):
    assert distill_fused(lib, **kw) == code


@pytest.mark.parametrize("kw,code", LOGITS + SPACE + DLOGITS + [
    (dict(lab=None), 1), (dict(adv=None), 1), (dict(ref=None), 1), (dict(options=None), 1)])
def test_policy_fused_refusals(lib, kw, code):
    assert policy_fused(lib, **kw) == code


@pytest.mark.parametrize("kw,code", SPACE + [
    (dict(lp=None), 1), (dict(adv=None), 1), (dict(ref=None), 1), (dict(options=None), 1), (dict(g=None), 1),
    (dict(rows=-1), 1), (dict(rows=1 << 30), 1), (dict(red=4), 1)])
def test_policy_refusals(lib, kw, code):
    assert policy(lib, **kw) == code


@pytest.mark.parametrize("kw", OPTIONS)
def test_policy_options_refused(lib, kw):
    assert policy(lib, policy_options(**kw)) == 1
    assert policy_fused(lib, policy_options(**kw)) == 1


@pytest.mark.parametrize("kw,code", LOGITS + SPACE + DLOGITS + [
    (dict(lab=None), 1), (dict(off=None), 1), (dict(pairs=0), 1), (dict(pairs=-1), 1), (dict(options=None), 1),
    (dict(pairs=1 << 31), 1)])
def test_preference_fused_refusals(lib, kw, code):
    assert preference_fused(lib, **kw) == code


@pytest.mark.parametrize("kw,code", SPACE + [
    (dict(lp=None), 1), (dict(off=None), 1), (dict(pairs=0), 1), (dict(options=None), 1), (dict(g=None), 1),
    (dict(rows=-1), 1), (dict(rows=1 << 30), 1), (dict(red=4), 1)])
def test_preference_refusals(lib, kw, code):
    assert preference(lib, **kw) == code


@pytest.mark.parametrize("kw", PAIRED)
def test_preference_options_refused(lib, kw):
    assert preference(lib, preference_options(**kw)) == 1
    assert preference_fused(lib, preference_options(**kw)) == 1


def test_calls_without_rows_still_want_their_loss(lib):
    assert distill_fwd(lib, rows=0, loss=None) == 1
    assert distill_fused(lib, rows=0, loss=None) == 1
    assert policy_fused(lib, rows=0, loss=None) == 1
    assert policy(lib, rows=0, loss=None) == 1
    assert distill_bwd(lib, rows=0, d=None, g=None, state=None) == 0


def test_workspace_size(lib):
    size = lib.gbce_preference_workspace_size
    assert size(-1, 2) == 0 and size(10, 0) == 0 and size(1 << 40, 2) == 0
    assert size(0, 1) > 0 and size(8192, 4) >= 8192 * 16 and size(8192, 4) < 8192 * 20


def test_python_refuses_cpu_tensors():
    import cross_entropy_gb300 as gbce

    x, i = torch.zeros((2, 8)), torch.zeros((2, 1), dtype=torch.int64)
    with pytest.raises(ValueError):
        gbce.distill_fwd(x, i, torch.zeros((2, 1)))
    with pytest.raises(ValueError):
        gbce.policy_loss(torch.zeros(2), torch.zeros(2))
    with pytest.raises(ValueError):
        gbce.policy_loss_fwd_bwd_fused(x, i[:, 0], torch.zeros(2))
    with pytest.raises(ValueError):
        gbce.preference_loss(torch.zeros(2), [0, 1, 2])
    with pytest.raises(ValueError):
        gbce.preference_loss_fwd_bwd_fused(x, i[:, 0], [0, 1, 2])
