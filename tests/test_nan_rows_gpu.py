"""Rows whose logits are all NaN, as a NaN hidden state gives them: every
output of theirs is NaN, and no other row's changes."""

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import cross_entropy_gb300 as gbce

DEV = "cuda:0"
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__

    __graft_entry__.build()
    gbce.load_library()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,V", [(3, 1), (3, 2), (5, 8), (700, 1000), (3, 152064), (400, 48000)])
def test_rows_of_nan_logits(rows, V, dtype):
    g = torch.Generator(device=DEV).manual_seed(V)
    clean = torch.randn((rows, V), generator=g, device=DEV).to(dtype)
    lab = torch.randint(0, V, (rows,), generator=g, device=DEV)
    idx = torch.stack([lab, (lab + V // 2) % V], 1)
    bad = torch.zeros(rows, dtype=torch.bool, device=DEV)
    bad[[0, rows - 1]] = True
    x = clean.clone()
    x[bad] = NAN
    one = torch.ones(rows, device=DEV)

    def calls(y):
        f = gbce.ce_fwd(y, lab, reduction="none")
        b = gbce.ce_bwd(y, lab, one, f.logp, reduction="none")
        u = gbce.ce_fwd_bwd_fused(y, lab, one, reduction="none")
        n = gbce.ce_fwd_bwd_fused_noalloc(y, lab, one, reduction="none")
        c = gbce.ce_fwd(y, lab, reduction="none", softcap=30.0)
        lp, ent = gbce.selective_logsoftmax(y, idx, with_entropy=True)
        only = gbce.selective_logsoftmax(y, idx)
        lb = gbce.selective_logsoftmax_bwd(y, idx, torch.ones_like(lp), lp)
        return dict(loss=f.loss, logp=f.logp, dlogits=b, fused=u.loss, fused_d=u.dlogits, capped=c.loss,
                    noalloc=n.loss, noalloc_d=n.dlogits, selective=only, with_entropy=lp, entropy=ent, selective_d=lb)

    for name, want in calls(clean).items():
        got = calls(x)[name]
        assert torch.isnan(got[bad]).all(), name
        assert torch.equal(got[~bad], want[~bad]) and torch.isfinite(want).all(), name
    assert torch.isnan(gbce.ce_fwd(x, lab).loss)
