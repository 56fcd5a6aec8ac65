"""The 64-bit forms the GPU tests compare with, held against differences and
against what the definitions say in special cases (CPU)."""

import math

import pytest
import torch

import post_ref as ref


def numeric(f, x, h=1e-6):
    g = torch.zeros_like(x)
    for i in range(x.numel()):
        a, b = x.clone(), x.clone()
        a.view(-1)[i] += h
        b.view(-1)[i] -= h
        g.view(-1)[i] = (f(a) - f(b)) / (2 * h)
    return g


@pytest.mark.parametrize("rest", [None, 0.4])
@pytest.mark.parametrize("T", [1.0, 0.6])
def test_distill_gradient_by_differences(rest, T):
    g = torch.Generator().manual_seed(3)
    x = torch.randn((1, 9), generator=g, dtype=torch.float64)
    idx = torch.tensor([[4, 0, -1, 7, 4]])
    t = torch.randn((1, 5), generator=g, dtype=torch.float64)
    r = None if rest is None else torch.tensor([rest]).double()
    loss, dz, _ = ref.distill(x, idx, t, r, T)
    num = numeric(lambda v: ref.distill(v, idx, t, r, T)[0][0], x)
    assert torch.allclose(dz / T, num, atol=1e-8)
    # the column listed twice: one entry with both probabilities
    merged = torch.tensor([[4, 0, 7]])
    tm = torch.stack([torch.logsumexp(t[0, [0, 4]] / T, 0) * T, t[0, 1], t[0, 3]]).unsqueeze(0)
    again, dz2, _ = ref.distill(x, merged, tm, r, T)
    assert torch.allclose(loss, again) and torch.allclose(dz, dz2)


def test_distill_is_kl_over_a_whole_vocabulary():
    g = torch.Generator().manual_seed(4)
    x, t = torch.randn((3, 6), generator=g).double(), torch.randn((3, 6), generator=g).double()
    idx = torch.arange(6).expand(3, 6)
    loss, dz, _ = ref.distill(x, idx, t, None, 1.0)
    want = torch.nn.functional.kl_div(x.log_softmax(1), t.log_softmax(1), reduction="none",
                                      log_target=True).sum(1)
    assert torch.allclose(loss, want)
    assert torch.allclose(dz, x.softmax(1) - t.softmax(1))
    # listing four of them, with the others' mass as the rest, bounds it from below
    part, dzp, _ = ref.distill(x, idx[:, :4], t[:, :4], torch.logsumexp(t[:, 4:], 1), 1.0)
    assert bool((part <= loss + 1e-12).all()) and torch.allclose(dzp.sum(1), torch.zeros(3).double())


@pytest.mark.parametrize("adv,move", [(1.5, 0.1), (1.5, 0.5), (-1.5, 0.1), (-1.5, -0.5), (0.0, 0.3)])
def test_policy_derivative_by_differences(adv, move):
    lp, a = torch.tensor([-1.3]).double(), torch.tensor([adv]).double()
    old, kl = lp - move, lp + 0.7
    _, d = ref.policy(lp, a, old, kl, 0.2, 0.28, 0.05)
    num = numeric(lambda v: ref.policy(v, a, old, kl, 0.2, 0.28, 0.05)[0][0], lp)
    assert torch.allclose(d, num, atol=1e-8)
    clamp = torch.exp(lp - old).clamp(0.8, 1.28)
    want = -torch.minimum(torch.exp(lp - old) * a, clamp * a) + 0.05 * (math.exp(0.7) - 0.7 - 1)
    assert torch.allclose(ref.policy(lp, a, old, kl, 0.2, 0.28, 0.05)[0], want)


@pytest.mark.parametrize("kind,eps,margin", [("sigmoid", 0.0, 0.0), ("sigmoid", 0.1, 0.5),
                                             ("squared", 0.0, 0.0)])
@pytest.mark.parametrize("average", [False, True])
def test_preference_derivative_by_differences(kind, eps, margin, average):
    g = torch.Generator().manual_seed(5)
    lp = -torch.rand(12, generator=g).double()
    kl = lp + 0.1 * torch.randn(12, generator=g).double()
    live = torch.rand(12, generator=g) < 0.8
    off = torch.tensor([1, 4, 4, 9, 11])
    args = (off, kl, live, 0.7, margin, eps, kind, average)
    _, _, d, _ = ref.preference(lp, *args)
    num = numeric(lambda v: ref.preference(v, *args)[0].sum(), lp)
    assert torch.allclose(d, num, atol=1e-8)
    assert d[0] == 0 and d[11] == 0
