"""The post-training losses at the sizes where another kernel or another number of warps takes the
rows: whole rows in shared memory (one, four and eight warps a row), streamed rows, rows split over a
cluster; bad input in each of them."""

import pytest
import torch

import post_ref as ref
import test_post_gpu as base
from test_post_gpu import BF16, DEV, F32, IGNORE, INF, NAN, NEG, gbce, gen, gpu, logits_of, teacher_of  # noqa: F401

pytestmark = pytest.mark.gpu

# rows, V, K, dtype, pad, shift: around 8 KB a row with more and with fewer than 400 rows, around 48 KB,
# around 104 KB with few rows (split) and with many, and around 1024 rows (who counts them)
SIZES = [(401, 4096, 33, BF16, 0, 0), (402, 4097, 7, BF16, 3, 1), (400, 2048, 32, F32, 0, 2),
         (1024, 65, 60, F32, 1, 1), (1027, 300, 256, BF16, 5, 3), (30, 24576, 200, BF16, 1, 5),
         (20, 24577, 256, BF16, 0, 0), (9, 53248, 64, BF16, 3, 3), (6, 53249, 64, BF16, 0, 1),
         (5, 26625, 130, F32, 2, 0), (240, 53255, 50, BF16, 7, 1), (17, 32769, 64, BF16, 3, 3),
         (16, 32769, 64, BF16, 0, 0), (40, 53248, 100, BF16, 1, 0), (18, 26624, 256, F32, 0, 1)]


@pytest.mark.parametrize("rows,V,K,dtype,pad,shift", SIZES)
@pytest.mark.parametrize("rest,ragged,T,reduction", [(True, True, 0.7, "mean"), (False, False, 1.0, "none")])
def test_distill(gbce, rows, V, K, dtype, pad, shift, rest, ragged, T, reduction):  # noqa: F811
    base.test_distill(gbce, rows, V, K, dtype, pad, shift, rest, ragged, T, reduction)


@pytest.mark.parametrize("rows,V,K,dtype,pad,shift", SIZES)
def test_policy(gbce, rows, V, K, dtype, pad, shift):  # noqa: F811
    base.test_policy(gbce, rows, V, dtype, pad, shift, 0.7, 0.1, "mean", True)


@pytest.mark.parametrize("rows,V,K,dtype,pad,shift", SIZES)
def test_preference(gbce, rows, V, K, dtype, pad, shift):  # noqa: F811
    base.test_preference(gbce, rows, V, 2, dtype, pad, 1, "sigmoid", True, True, "mean", 2.0, 0.1, 0.5)


@pytest.mark.parametrize("rows,V,dtype", [(500, 3001, BF16), (500, 700, F32), (9, 20001, BF16), (9, 40001, BF16), (30, 40001, BF16),
                                          (9, 60001, BF16), (240, 60001, BF16), (240, 27001, F32)])
def test_bad_rows_among_good_ones(gbce, rows, V, dtype):  # noqa: F811
    g = gen(V + rows)
    x = logits_of(rows, V, dtype, g)
    idx, t, r = teacher_of(x, 40, g, False, True)
    idx[0, 35] = idx[0, 1]            # one column named twice, and one four times (over two warps)
    idx[1, 3] = idx[1, 37] = idx[1, 11] = idx[1, 2]
    idx[2, 39] = V                    # outside the vocabulary
    t[3, 6] = NAN
    idx[4], r[4] = -1, NEG            # nothing at all
    x[5, idx[5, 3]] = NAN             # no softmax
    idx[6] = -1                       # a rest alone
    per, dz, move = ref.distill(x.float(), idx, t, r, 1.3)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    xg, args = gpu(x), (gpu(idx), gpu(t), gpu(r))
    one = torch.ones(rows, device=DEV)
    out = gbce.distill_fwd_bwd_fused(xg, *args, one, 1.3, None, "none", dev_status=flag)
    f = gbce.distill_fwd(xg, *args, 1.3, None, "none", dev_status=flag)
    b = gbce.distill_bwd(xg, *args, one, f.rest_state, None, 1.3, None, "none", dev_status=flag)
    assert int(flag) == 2
    for loss, d in ((out.loss, out.dlogits), (f.loss, b)):
        for bad in (2, 3, 5):
            assert bool(torch.isnan(loss[bad])) and bool(torch.isnan(d[bad]).all()), bad
        assert float(loss[4]) == 0 and not bool(d[4].any())
        good = [i for i in range(min(rows, 16)) if i not in (2, 3, 5)] + [rows - 1]
        base.close(loss[good], per[good], base.LOSS_TOL,
                   ref.kl_bound(per[good], move[:, good]).nan_to_num(0.0, 0.0, 0.0))
        base.rows_close(d[good], dz[good] / 1.3, dtype, floor=ref.gap_bound(move[:, good]) / 1.3)
    # a label outside the vocabulary, one left out, a NaN logit
    lab = torch.randint(0, V, (rows,), generator=g)
    lab[0], lab[1], lab[2] = V, IGNORE, -7
    x = logits_of(rows, V, dtype, g)
    x[3, 5] = NAN
    x[1] = NAN
    flag.zero_()
    p = gbce.policy_loss_fwd_bwd_fused(gpu(x), gpu(lab), one, None, None, one, reduction="none", dev_status=flag)
    assert int(flag) == 1
    for i, nan in ((0, True), (1, False), (2, True), (3, True), (4, False)):
        assert bool(torch.isnan(p.loss[i])) == nan and bool(torch.isnan(p.dlogits[i]).any()) == nan, i
        assert bool(torch.isnan(p.dlogits[i]).all()) == nan, i
    assert not bool(p.dlogits[1].any()) and float(p.logp[1]) == 0


@pytest.mark.parametrize("rows,V,dtype", [(1500, 53300, BF16), (800, 53300, F32)])
def test_left_out_rows_change_no_streamed_row(gbce, rows, V, dtype):  # noqa: F811
    """Several streamed rows per CTA: a kept row has the same bits whatever rows lie between."""
    g = torch.Generator(device=DEV).manual_seed(V)
    x = (torch.randn((rows, V), generator=g, device=DEV) * 2.0).to(dtype)
    idx = torch.randint(0, V // 8, (rows, 8), generator=g, device=DEV) + torch.arange(8, device=DEV) * (V // 8)
    t = torch.randn((rows, 8), generator=g, device=DEV) + 6.0
    one = torch.ones(rows, device=DEV)
    whole = gbce.distill_fwd_bwd_fused(x, idx, t, None, one, 1.0, None, "none")
    for share in (0.2, 0.5, 0.9):
        mask = (torch.rand(rows, generator=g, device=DEV) >= share).to(torch.uint8)
        out = gbce.distill_fwd_bwd_fused(x, idx, t, None, one, 1.0, mask, "none")
        kept = mask.bool()
        assert torch.equal(out.loss[kept], whole.loss[kept]) and torch.equal(out.dlogits[kept], whole.dlogits[kept])
        assert not bool(out.dlogits[~kept].any()) and int(out.n_items) == int(kept.sum())


def test_a_coefficient_held_in_a_tensor(gbce):  # noqa: F811
    """A coefficient that changes in place (a schedule kept as a tensor) is read at every call."""
    g = gen(3)
    lp, kl, adv = (torch.randn(40, generator=g) for _ in range(3))
    beta = torch.tensor(0.0)
    for value in (0.0, 0.5, 2.0):
        beta.fill_(value)
        got = gbce.policy_loss(gpu(lp), gpu(adv), None, gpu(kl), kl_beta=beta)
        want = gbce.policy_loss(gpu(lp), gpu(adv), None, gpu(kl), kl_beta=value)
        assert torch.equal(got.loss, want.loss) and torch.equal(got.dlogp, want.dlogp)
    first = None
    for value in (0.1, 0.4):
        beta.fill_(value)
        got = gbce.preference_loss(gpu(lp), [0, 20, 40], beta=beta).loss
        assert torch.equal(got, gbce.preference_loss(gpu(lp), [0, 20, 40], beta=value).loss)
        assert first is None or not torch.equal(got, first)
        first = got


@pytest.mark.parametrize("rows,V", [(5000, 700), (300, 9000), (300, 40000)])
def test_the_same_bits_in_a_graph_beside_eager_calls(gbce, rows, V):  # noqa: F811
    g = gen(V)
    x = gpu(logits_of(rows, V, BF16, g))
    lab, adv = gpu(torch.randint(0, V, (rows,), generator=g)), gpu(torch.randn(rows, generator=g))
    lab[::3] = IGNORE
    off = gpu(torch.tensor([0, rows // 2, rows]))

    def step():
        p = gbce.policy_loss_fwd_bwd_fused(x, lab, adv)
        q = gbce.preference_loss_fwd_bwd_fused(x, lab, off, average=True)
        return p.loss, p.dlogits, p.n_items, q.loss, q.dlogits, q.seq_score

    want = [v.clone() for v in step()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        graph.replay()
        with torch.cuda.stream(side):
            other = step()
    torch.cuda.synchronize()
    for a, b, w in zip(held, other, want):
        assert torch.equal(a, w) and torch.equal(b, w)


@pytest.mark.parametrize("rows,V,K", [(402, 1, 3), (402, 90, 256), (7, 90, 256), (20, 30000, 256), (230, 60000, 256)])
def test_lists_of_one_column(gbce, rows, V, K):  # noqa: F811
    """Every entry names the same column, or one of two: their teacher's sums in entry order."""
    g = gen(V + K)
    x = logits_of(rows, V, F32 if V < 100 else BF16, g)
    idx = torch.full((rows, K), V - 1)
    idx[::2, ::3] = 0
    t = torch.randn((rows, K), generator=g)
    r = torch.randn(rows, generator=g) if V > 2 else None
    base.distill_check(gbce, x, idx, t, r, 0.9, None, "mean", seed=V)
