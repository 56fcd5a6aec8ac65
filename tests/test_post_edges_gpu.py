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
