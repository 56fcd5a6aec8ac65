"""Host-side checks of the linear_* and embedding_* calls: every refusal
returns before any CUDA call, so none of this needs a GPU."""

import pytest


@pytest.fixture(scope="module")
def lib():
    from cross_entropy_gb300 import build

    path = build.build()
    import cross_entropy_gb300 as gbce

    return gbce.load_library(path)


P = 0x100000  # never dereferenced
BIG = 1 << 40


def far(i):
    """Addresses that do not overlap for these sizes."""
    return P + i * (1 << 24)


def sel(lib, **kw):
    a = dict(h=far(0), hs=64, w=far(1), ws=64, dtype=1, rows=4, vocab=100, dim=64, idx=far(2), k=1,
             T=1.0, mask=None, out=far(3), state=None, wk=far(4), wb=BIG, st=None, s=None)
    a.update(kw)
    return lib.linear_selective_logsoftmax(*a.values())


def bwd(lib, **kw):
    a = dict(h=far(0), hs=64, w=far(1), ws=64, dtype=1, rows=4, vocab=100, dim=64, idx=far(2), k=1,
             T=1.0, mask=None, g=far(5), lp=far(6), rs=far(7), dh=far(8), dhs=64, dw=far(9), dws=64,
             acc=0, wk=far(4), wb=BIG, st=None, s=None)
    a.update(kw)
    return lib.linear_selective_logsoftmax_bwd(*a.values())


def fused(lib, **kw):
    a = dict(h=far(0), hs=64, w=far(1), ws=64, dtype=1, rows=4, vocab=100, dim=64, lab=far(2),
             ign=-100, T=1.0, red=2, g=far(5), loss=far(6), lp=None, rs=None, n=None, dh=far(8),
             dhs=64, dw=far(9), dws=64, acc=0, wk=far(4), wb=BIG, st=None, s=None)
    a.update(kw)
    return lib.linear_ce_fwd_bwd_fused(*a.values())


SHAPE = [
    (dict(dtype=7), 2), (dict(h=far(0) + 1), 2), (dict(w=far(1) + 1), 2), (dict(h=None), 1),
    (dict(w=None), 1), (dict(hs=63), 1), (dict(ws=63), 1), (dict(rows=-1), 1),
    (dict(rows=(1 << 24) + 1), 1), (dict(vocab=0), 1), (dict(vocab=1 << 31), 1), (dict(dim=0), 1),
    (dict(dim=(1 << 20) + 1), 1), (dict(T=0.0), 1), (dict(T=float("nan")), 1),
    (dict(wk=None), 4), (dict(wk=far(4) + 8), 4), (dict(wk=far(4) + 16), 4), (dict(wb=64), 4),
]


@pytest.mark.parametrize("kw,code", SHAPE + [(dict(k=0), 1), (dict(k=17), 1), (dict(idx=None), 1),
                                             (dict(out=None), 1)])
def test_selective_refusals(lib, kw, code):
    assert sel(lib, **kw) == code


GRADS = [
    (dict(dh=None, dw=None), 1), (dict(dhs=63), 1), (dict(dws=63), 1), (dict(dh=far(8) + 1), 2),
    (dict(dh=far(0)), 1), (dict(dh=far(1) + 128), 1), (dict(dw=far(1)), 1), (dict(dw=far(0)), 1),
    (dict(dw=far(8)), 1), (dict(g=None), 1),
]


@pytest.mark.parametrize("kw,code", SHAPE + GRADS + [(dict(lp=None), 1), (dict(rs=None), 1),
                                                     (dict(k=17), 1), (dict(idx=None), 1)])
def test_selective_backward_refusals(lib, kw, code):
    assert bwd(lib, **kw) == code


@pytest.mark.parametrize("kw,code", SHAPE + GRADS + [(dict(lab=None), 1), (dict(loss=None), 1),
                                                     (dict(red=5), 1), (dict(red=-1), 1)])
def test_fused_refusals(lib, kw, code):
    assert fused(lib, **kw) == code


def test_ce_backward_mean_needs_n_items(lib):
    a = [far(0), 64, far(1), 64, 1, 4, 100, 64, far(2), -100, 1.0, 2, far(5), far(6), far(7), None,
         far(8), 64, far(9), 64, 0, far(4), BIG, None, None]
    assert lib.linear_ce_bwd(*a) == 1


def test_workspace_sizes(lib):
    size = lib.gbce_linear_workspace_size
    assert size(0, 100, 64, 1, 1, 1) == 0 and size(4, 0, 64, 1, 1, 1) == 0
    assert size(4, 100, 64, 17, 1, 1) == 0 and size(4, 100, 64, 1, 9, 1) == 0
    assert 0 < size(4, 100, 64, 1, 1, 0) < size(4, 100, 64, 1, 1, 1)
    # far from the logits' size: the vocabulary goes by in pieces
    logits = 8192 * 152064 * 2
    assert size(8192, 152064, 4096, 1, 1, 1) < logits // 2
    assert size(8192, 152064, 4096, 1, 1, 0) < logits // 8
    assert lib.gbce_embedding_workspace_size(0, 10, 10) == 0
    assert lib.gbce_embedding_workspace_size(100, 10, 10) > 0


def lookup(lib, **kw):
    a = dict(t=far(0), ts=64, dtype=1, vocab=100, dim=64, tok=far(1), rows=4, ign=-100, scale=1.0,
             out=far(2), os=64, st=None, s=None)
    a.update(kw)
    return lib.embedding_lookup(*a.values())


def lookup_bwd(lib, **kw):
    a = dict(g=far(0), gs=64, dtype=1, rows=4, dim=64, tok=far(1), vocab=100, ign=-100, scale=1.0,
             d=far(2), ds=64, acc=0, wk=far(3), wb=BIG, st=None, s=None)
    a.update(kw)
    return lib.embedding_lookup_bwd(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), 2), (dict(t=None), 1), (dict(ts=63), 1), (dict(t=far(0) + 1), 2),
    (dict(vocab=0), 1), (dict(dim=0), 1), (dict(rows=-1), 1), (dict(scale=float("inf")), 1),
    (dict(scale=float("nan")), 1), (dict(tok=None), 1), (dict(out=None), 1), (dict(os=1), 1),
    (dict(out=far(0) + 64), 1),
])
def test_lookup_refusals(lib, kw, code):
    assert lookup(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), 2), (dict(g=None), 1), (dict(gs=63), 1), (dict(g=far(0) + 1), 2),
    (dict(vocab=0), 1), (dict(dim=0), 1), (dict(rows=-1), 1), (dict(scale=float("nan")), 1),
    (dict(tok=None), 1), (dict(d=None), 1), (dict(ds=1), 1), (dict(d=far(0)), 1),
    (dict(wk=None), 4), (dict(wk=far(3) + 4), 4), (dict(wb=0), 4),
])
def test_lookup_gradient_refusals(lib, kw, code):
    assert lookup_bwd(lib, **kw) == code


def test_binding_refuses_what_it_cannot_marshal():
    import torch

    import cross_entropy_gb300 as gbce

    h, w = torch.zeros(2, 8), torch.zeros(5, 8)
    lab = torch.zeros(2, dtype=torch.int64)
    for call in (lambda: gbce.linear_ce_fwd(h, w, lab),
                 lambda: gbce.linear_ce_fwd_bwd_fused(h, w, lab),
                 lambda: gbce.linear_selective_logsoftmax(h, w, lab),
                 lambda: gbce.embedding_lookup(w, lab),
                 lambda: gbce.embedding_lookup_bwd(h, lab, 5)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="accumulate"):
        gbce.linear_ce_fwd_bwd_fused(h, w, lab, accumulate=True)
    with pytest.raises(TypeError):
        gbce.linear_workspace_size(1, 1, 1, dtype=torch.float16)
