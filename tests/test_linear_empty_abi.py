"""Refusals of linear calls without rows: what they would write, and beside
what, is checked as for any other call (all of it before any CUDA call, so
none of this needs a GPU)."""

import pytest

from test_linear_abi import bwd, far, fused, lib, sel  # noqa: F401


def ce_bwd(lib, **kw):
    a = dict(h=far(0), hs=64, w=far(1), ws=64, dtype=1, rows=4, vocab=100, dim=64, lab=far(2),
             ign=-100, T=1.0, red=1, g=far(5), lp=far(6), rs=far(7), n=None, dh=far(8), dhs=64,
             dw=far(9), dws=64, acc=0, wk=far(4), wb=1 << 40, st=None, s=None)
    a.update(kw)
    return lib.linear_ce_bwd(*a.values())


@pytest.mark.parametrize("call", [bwd, fused, ce_bwd])
@pytest.mark.parametrize("kw,code", [
    (dict(dh=None, dw=None), 1),           # nothing wanted
    (dict(hs=63), 1), (dict(ws=63), 1), (dict(dhs=63), 1), (dict(dws=63), 1),
    (dict(dw=far(9) + 1), 2), (dict(w=far(1) + 1), 2), (dict(w=None), 1),
    (dict(dw=far(1)), 1),                  # zeros would go over the weight
    (dict(dw=far(1) + 64 * 99 * 2), 1),    # over its last row
])
def test_gradient_calls_without_rows(lib, call, kw, code):  # noqa: F811
    assert call(lib, rows=0, **kw) == code


def test_forward_without_rows(lib):  # noqa: F811
    assert sel(lib, rows=0, h=None, idx=None, out=None, wk=None, wb=0) == 0
    assert sel(lib, rows=0, hs=63) == 1 and sel(lib, rows=0, ws=63) == 1


def test_empty_gradients_overlap_nothing(lib):  # noqa: F811
    # accumulating or unwanted, dweight is not written, so these return before
    # any CUDA call
    for call in (bwd, ce_bwd):
        assert call(lib, rows=0, h=None, dh=far(1), dw=far(9), acc=1) == 0
        assert call(lib, rows=0, h=None, dh=far(9) + 128, dw=far(9), acc=1) == 0
        assert call(lib, rows=0, h=None, dh=far(1), dw=None) == 0
