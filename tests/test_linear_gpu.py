"""linear_selective_logsoftmax, linear_ce_* and their gradients against the
definitions in 64 bits: odd sizes, strides, masks, duplicates, bad targets,
streams, graphs and poisoned workspaces."""

import math

import numpy as np
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import cross_entropy_gb300 as gbce

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__

    __graft_entry__.build()
    gbce.load_library()


def strided(t, pad, shift=0):
    """The same values as rows of a wider buffer, `shift` elements into it."""
    n, d = t.shape
    buf = torch.full((n * (d + pad) + shift,), math.nan, dtype=t.dtype, device=t.device)
    view = buf[shift:].view(n, d + pad)[:, :d]
    view.copy_(t)
    return view


def problem(rows, V, D, K, dtype, seed, margin=True, std=2.5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = (torch.randn((V, D), generator=g, device=DEV) * (std / math.sqrt(D))).to(dtype)
    t = torch.randint(0, V, (rows, K), generator=g, device=DEV)
    if K > 2 and rows:
        t[::3, 2] = t[::3, 0]
    h = torch.randn((rows, D), generator=g, device=DEV)
    if margin and rows and D > 8:
        wt = w[t[:, 0]].float()
        lead = torch.rand(rows, generator=g, device=DEV) * 45.0
        lead[::2] = 0.0
        h += (lead / wt.square().sum(1).clamp(min=1e-3))[:, None] * wt
    mask = (torch.rand(rows, generator=g, device=DEV) > 0.2).to(torch.uint8)
    up = torch.randn((rows, K), generator=g, device=DEV) / max(rows, 1)
    return h.to(dtype), w, t, mask, up


def check_selective(h, w, t, mask, up, T, logp, dh=None, dw=None):
    rows, K = t.shape
    live = mask.bool() if mask is not None else torch.ones(rows, dtype=torch.bool, device=DEV)
    p, lp, comp, ez = ref.rows_of(h, w, t, T, live)
    full = torch.zeros((rows, K), dtype=torch.float64, device=DEV)
    full[live] = lp
    b = torch.zeros_like(full)
    b[live] = ref.logp_bound(lp, comp, ez)
    ref.assert_within(logp, full, b, "log p")
    assert not (logp > 0).any()
    if dh is None:
        return
    dz, size = ref.selective_dz(p, lp, comp, t[live], up[live].double(), T)
    hl, wd = h[live].double(), w.double()
    rdh, rdw, bh, bw = ref.products(dz, size, hl, wd, ez, h.dtype)
    fdh = torch.zeros(h.shape, dtype=torch.float64, device=DEV)
    fdh[live] = rdh
    fb = torch.zeros_like(fdh)
    fb[live] = bh
    ref.assert_within(dh, fdh, fb, "dhidden")
    ref.assert_within(dw, rdw, bw, "dweight")


SIZES = [  # rows, vocab, dim, K
    (1, 1, 1, 1), (1, 2, 3, 1), (2, 1, 8, 2), (3, 257, 8, 16), (1, 4096, 64, 1), (5, 255, 63, 3),
    (127, 1003, 65, 1), (128, 256, 64, 2), (129, 513, 72, 4), (255, 300, 200, 1),
    (257, 1000, 129, 5), (300, 19457, 96, 2), (64, 40001, 136, 1), (513, 777, 1001, 3),
    (1025, 2049, 264, 1),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,V,D,K", SIZES)
def test_selective_step_against_64_bits(rows, V, D, K, dtype):
    T = 0.9
    h, w, t, mask, up = problem(rows, V, D, K, dtype, rows * 7 + V)
    logp, state = gbce.linear_selective_logsoftmax(h, w, t, T, mask, with_state=True)
    dh, dw = gbce.linear_selective_logsoftmax_bwd(h, w, t, up, logp, state, T, mask)
    check_selective(h, w, t, mask, up, T, logp, dh, dw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
@pytest.mark.parametrize("rows,V,D", [(1, 4096, 64), (77, 1003, 200), (300, 5000, 256)])
def test_ce_fused_equals_its_parts_and_64_bits(rows, V, D, reduction, dtype):
    T = 1.3
    h, w, t, mask, up = problem(rows, V, D, 1, dtype, rows + V)
    if rows > 1:
        mask[0] = 1
    lab = torch.where(mask.bool(), t[:, 0], torch.full_like(t[:, 0], -100))
    g = torch.rand(rows if reduction == "none" else 1, device=DEV) + 0.5
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = gbce.linear_ce_fwd_bwd_fused(h, w, lab, g, temperature=T, reduction=reduction,
                                       want_logp=True, dev_status=st)
    f = gbce.linear_ce_fwd(h, w, lab, temperature=T, reduction=reduction)
    dh, dw = gbce.linear_ce_bwd(h, w, lab, g, f.logp, f.row_state, f.n_items, temperature=T,
                                reduction=reduction)
    assert torch.equal(out.loss, f.loss) and torch.equal(out.logp, f.logp)
    assert torch.equal(out.dhidden, dh) and torch.equal(out.dweight, dw)
    live = mask.bool()
    n = int(live.sum())
    assert int(out.n_items) == n and int(st) == 0
    check_selective(h, w, lab[:, None].clamp(min=0), mask, None, T, f.logp[:, None])
    per = -f.logp.double()
    want = {"none": per, "sum": per.sum(), "mean": per.sum() / max(n, 1)}[reduction]
    ref.assert_within(out.loss, want, want.abs() * 2 ** -23, "loss")
    # u_r = -upstream of log p
    up = -(g.expand(rows)[:, None] / (n if reduction == "mean" and n else 1)).double()
    check_selective(h, w, lab[:, None].clamp(min=0), mask, up, T, f.logp[:, None], dh, dw)


def test_all_rows_left_out_and_no_rows():
    w = torch.randn((300, 64), device=DEV, dtype=torch.bfloat16)
    h = torch.full((5, 64), math.nan, device=DEV, dtype=torch.bfloat16)
    lab = torch.full((5,), -100, device=DEV)
    out = gbce.linear_ce_fwd_bwd_fused(h, w, lab, dweight=torch.full_like(w, 7.0))
    assert out.loss == 0 and int(out.n_items) == 0
    assert not out.dhidden.any() and not out.dweight.any()
    keep = torch.full_like(w, 7.0)
    gbce.linear_ce_fwd_bwd_fused(h, w, lab, dweight=keep, accumulate=True)
    assert (keep == 7.0).all()
    empty = gbce.linear_ce_fwd_bwd_fused(h[:0], w, lab[:0], dweight=torch.full_like(w, 7.0))
    assert empty.loss == 0 and int(empty.n_items) == 0 and not empty.dweight.any()
    assert empty.dhidden.shape == (0, 64)
    logp = gbce.linear_selective_logsoftmax(h, w, torch.zeros((5, 2), dtype=torch.int64), 1.0,
                                            torch.zeros(5, dtype=torch.uint8))
    assert logp.shape == (5, 2) and not logp.any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_what_left_out_rows_hold_does_not_matter(dtype):
    h, w, t, mask, up = problem(300, 700, 96, 2, dtype, 5)
    mask[0] = mask[-1] = 0
    dirty = h.clone()
    dirty[mask == 0] = math.nan
    dirty[0] = math.inf
    runs = []
    for x in (h, dirty):
        logp, state = gbce.linear_selective_logsoftmax(x, w, t, 1.0, mask, with_state=True)
        runs.append((logp, *gbce.linear_selective_logsoftmax_bwd(x, w, t, up, logp, state, 1.0, mask)))
    for a, b in zip(*runs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("pads", [(0, 0, 0, 1), (8, 0, 8, 0), (3, 5, 1, 0), (8, 8, 8, 8)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_and_misaligned_operands_and_outputs(dtype, pads):
    hp, wp, gp, shift = pads
    h, w, t, mask, up = problem(131, 515, 88, 1, dtype, 3)
    base = gbce.linear_ce_fwd_bwd_fused(h, w, t[:, 0])
    dh = strided(torch.zeros_like(h), gp, shift)
    dw = strided(torch.zeros_like(w), gp, shift)
    out = gbce.linear_ce_fwd_bwd_fused(strided(h, hp, shift), strided(w, wp, shift), t[:, 0],
                                       dhidden=dh, dweight=dw)
    for a, b in zip(base[:3], out[:3]):
        assert torch.equal(a, b)
    for d in (dh, dw):  # the gaps between rows stay as they were
        whole = torch.as_strided(d, (d.shape[0] - 1, gp), (d.stride(0), 1),
                                 d.storage_offset() + d.shape[1])
        assert torch.isnan(whole).all()


@pytest.mark.parametrize("rows", [1, 5, 128, 129])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_short_forwards_in_place_and_packed_agree(rows, pad):
    # up to 128 rows that start on 16 bytes are read where they are: the same
    # bits as from a packed copy, with masked, ignored and bad targets sorted out
    h, w, t, mask, up = problem(rows, 777, 96, 3, torch.bfloat16, rows)
    if rows > 2:
        mask[1] = 0
        h[1] = math.nan
    logp, state = gbce.linear_selective_logsoftmax(strided(h, pad), w, t, 0.9, mask, with_state=True)
    base, bstate = gbce.linear_selective_logsoftmax(strided(h, 3), w, t, 0.9, mask, with_state=True)
    assert torch.equal(logp, base) and torch.equal(state, bstate)
    check_selective(torch.nan_to_num(h), w, t, mask, None, 0.9, logp)
    lab = t[:, 0].clone()
    lab[0] = 777 if rows > 4 else lab[0]
    if rows > 2:
        lab[2] = -100
    for red in ("none", "sum", "mean"):
        st = torch.zeros(2, dtype=torch.int32, device=DEV)
        a = gbce.linear_ce_fwd(strided(h, pad), w, lab, reduction=red, dev_status=st[:1])
        b = gbce.linear_ce_fwd(strided(h, 3), w, lab, reduction=red, dev_status=st[1:])
        for x, y in zip(a, b):
            assert torch.equal(torch.nan_to_num(x, 7.0), torch.nan_to_num(y, 7.0))
        assert int(st[0]) == int(st[1]) == (gbce.DEV_BAD_LABEL if rows > 4 else 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,D,pad", [(1, 4096, 0), (48, 4096, 8), (300, 4096, 0), (300, 4095, 0), (700, 2561, 3)])
def test_confident_rows_keep_their_digits(rows, D, pad, dtype):
    # One column of weight, the others zero: their logits are exactly 0 and log p
    # = -softplus(log(V - 1) - z), whose relative error is what z and the steps
    # after it are off by.  All products of z are positive, so in 256 running
    # sums of D / 256 terms and a tree of 8 levels it carries at most
    # (D / 512 + 1 + 8) u z (half a sum on average, one half ulp a term); the
    # temperature, the log, the differences and exp2's argument 6 u (z + 12)
    # more, exp2 and log1p 16 u.  Sums that are cut instead of rounded, 64
    # steps long and more, are off by 64 u z and more.
    g = torch.Generator(device=DEV).manual_seed(D + rows)
    V, at = 513, 300
    w = torch.zeros((V, D), dtype=dtype, device=DEV)
    w[at] = (torch.rand(D, generator=g, device=DEV) + 0.5).to(dtype)
    lead = 20.0 + 40.0 * torch.rand(rows, 1, generator=g, device=DEV)
    h = (lead * w[at].float() / w[at].float().square().sum()).to(dtype)
    lab = torch.full((rows,), at, dtype=torch.int64, device=DEV)
    z = h.double() @ w[at].double()
    exp = -torch.nn.functional.softplus(math.log(V - 1) - z, threshold=1e9)
    bound = exp.abs() * (ref.U * ((D / 512 + 9) * z + 6 * (z + 12) + 16))
    logp, _ = gbce.linear_selective_logsoftmax(strided(h, pad), strided(w, pad), lab[:, None], 1.0, with_state=True)
    ref.assert_within(logp[:, 0], exp, bound, "log p")
    both = gbce.linear_ce_fwd_bwd_fused(strided(h, pad), strided(w, pad), lab, want_logp=True)
    assert torch.equal(both.logp.reshape(-1), logp[:, 0])


def test_more_rows_than_a_grid_axis_takes():
    # kept logits of 70000 rows
    h, w, t, mask, up = problem(70000, 64, 16, 1, torch.bfloat16, 31)
    lab = torch.where(mask.bool(), t[:, 0], torch.full_like(t[:, 0], -100))
    out = gbce.linear_ce_fwd_bwd_fused(h, w, lab, reduction="sum", want_logp=True)
    f = gbce.linear_ce_fwd(h, w, lab, reduction="sum")
    dh, dw = gbce.linear_ce_bwd(h, w, lab, torch.ones(1), f.logp, f.row_state, f.n_items, reduction="sum")
    assert torch.equal(out.dhidden, dh) and torch.equal(out.dweight, dw) and torch.equal(out.logp, f.logp)
    check_selective(h, w, lab[:, None].clamp(min=0), mask, -torch.ones((70000, 1), device=DEV), 1.0,
                    f.logp[:, None], dh, dw)


@pytest.mark.parametrize("rows,V,D,K,dtype", [
    (4000, 60001, 64, 2, torch.bfloat16),    # two pieces, the last one ragged
    (3900, 40001, 40, 1, torch.float32),     # three pieces
    (8, 40001, 4600, 1, torch.float32),      # a weight packed in parts
    (100, 40001, 4601, 3, torch.bfloat16),   # the same, rows that do not start on 16 bytes
])
def test_vocabularies_of_several_pieces(rows, V, D, K, dtype):
    h, w, t, mask, up = problem(rows, V, D, K, dtype, V + D)
    logp, state = gbce.linear_selective_logsoftmax(h, w, t, 0.9, mask, with_state=True)
    dh, dw = gbce.linear_selective_logsoftmax_bwd(h, w, t, up, logp, state, 0.9, mask)
    check_selective(h, w, t, mask, up, 0.9, logp, dh, dw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shift", [0, 1])
def test_exact_workspace_for_any_alignment_of_the_weight(dtype, shift):
    h, w, t, mask, up = problem(260, 20011, 88, 1, dtype, 33)
    x = strided(w, 1 if shift else 0, shift)
    n = gbce.linear_workspace_size(260, 20011, 88, 1, dtype)
    guard = torch.full((n + 4096,), 173, dtype=torch.uint8, device=DEV)
    out = gbce.linear_ce_fwd_bwd_fused(h, x, t[:, 0], workspace=guard[:n])
    again = gbce.linear_ce_fwd_bwd_fused(h, w, t[:, 0])
    for a, b in zip(again[:3], out[:3]):
        assert torch.equal(a, b)
    assert (guard[n:] == 173).all()
    with pytest.raises(gbce.GbceError):
        gbce.linear_ce_fwd_bwd_fused(h, x, t[:, 0], workspace=guard[:n - 256])


def test_three_dimensional_hidden_and_single_index():
    h, w, t, mask, up = problem(24, 300, 64, 1, torch.bfloat16, 9)
    flat, st = gbce.linear_selective_logsoftmax(h, w, t[:, 0], with_state=True)
    out = gbce.linear_selective_logsoftmax(h.view(2, 12, 64), w, t.view(2, 12, 1))
    assert out.shape == (2, 12, 1) and torch.equal(out.view(-1), flat)
    dh, _ = gbce.linear_selective_logsoftmax_bwd(h.view(2, 12, 64), w, t.view(2, 12), up.view(2, 12),
                                                 flat.view(2, 12), st)
    assert dh.shape == (2, 12, 64)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_accumulating_and_unwanted_gradients(dtype):
    h, w, t, mask, up = problem(200, 600, 72, 1, dtype, 11)
    ref_out = gbce.linear_ce_fwd_bwd_fused(h, w, t[:, 0])
    start = torch.randn_like(w.float()).to(dtype) * 0.01
    acc = start.clone()
    out = gbce.linear_ce_fwd_bwd_fused(h, w, t[:, 0], dweight=acc, accumulate=True,
                                       want_dhidden=False)
    assert out.dhidden is None and out.dweight is acc
    # added in fp32 and rounded once: within half a step of the sum, and of the
    # fresh gradient's own rounding
    want = start.double() + ref_out.dweight.double()
    half = ref.HALF[dtype]
    ref.assert_within(acc, want, half * (want.abs() + 2 * ref_out.dweight.double().abs()) + 1e-30, "sum")
    only = gbce.linear_ce_fwd_bwd_fused(h, w, t[:, 0], want_dweight=False)
    assert only.dweight is None and torch.equal(only.dhidden, ref_out.dhidden)
    with pytest.raises(gbce.GbceError):
        gbce.linear_ce_fwd_bwd_fused(h, w, t[:, 0], want_dweight=False, want_dhidden=False)


def test_bad_labels_and_indices():
    h, w, t, mask, up = problem(40, 500, 64, 2, torch.bfloat16, 13)
    lab = t[:, 0].clone()
    lab[3], lab[7], lab[9] = 500, -1, -100
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = gbce.linear_ce_fwd_bwd_fused(h, w, lab, reduction="none", want_logp=True, dev_status=st)
    assert int(st) == gbce.DEV_BAD_LABEL
    bad = torch.zeros(40, dtype=torch.bool, device=DEV)
    bad[[3, 7]] = True
    assert torch.isnan(out.loss[bad]).all() and torch.isnan(out.dhidden[bad]).all()
    assert torch.isfinite(out.loss[~bad]).all() and torch.isfinite(out.dhidden[~bad]).all()
    assert int(out.n_items) == 39 and out.loss[9] == 0
    keep = lab.clone()
    keep[bad] = -100  # the rows are left out of dweight
    assert torch.equal(out.dweight, gbce.linear_ce_fwd_bwd_fused(h, w, keep, reduction="none").dweight)
    mean = gbce.linear_ce_fwd(h, w, lab)
    assert torch.isnan(mean.loss) and int(mean.n_items) == 39
    t[5, 1] = 1 << 40
    st.zero_()
    logp, state = gbce.linear_selective_logsoftmax(h, w, t, with_state=True, dev_status=st)
    assert int(st) == gbce.DEV_BAD_INDEX and torch.isnan(logp[5, 1])
    assert int(torch.isnan(logp).sum()) == 1 and torch.isfinite(state).all()
    st.zero_()
    dh, dw = gbce.linear_selective_logsoftmax_bwd(h, w, t, up, logp, state, dev_status=st)
    assert int(st) == gbce.DEV_BAD_INDEX and torch.isnan(dh[5]).all()
    assert torch.isfinite(dw).all() and int(torch.isnan(dh).any(1).sum()) == 1


def test_nan_and_inf_in_a_live_row_stay_in_it():
    h, w, t, mask, up = problem(150, 400, 64, 1, torch.bfloat16, 15)
    clean = gbce.linear_selective_logsoftmax(h, w, t)
    h[17, 3] = math.nan
    h[100, 0] = math.inf
    logp = gbce.linear_selective_logsoftmax(h, w, t)
    assert torch.isnan(logp[17]).all()
    keep = torch.ones(150, dtype=torch.bool, device=DEV)
    keep[[17, 100]] = False
    assert torch.equal(logp[keep], clean[keep])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_same_bits_again_in_a_poisoned_workspace(dtype):
    h, w, t, mask, up = problem(515, 3001, 104, 3, dtype, 17)
    need = gbce.linear_workspace_size(515, 3001, 104, 3, dtype)
    outs = []
    for fill in (0, 255):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=DEV)
        logp, state = gbce.linear_selective_logsoftmax(h, w, t, 0.7, mask, with_state=True, workspace=ws)
        ws.fill_(fill)
        outs.append((logp, state, *gbce.linear_selective_logsoftmax_bwd(
            h, w, t, up, logp, state, 0.7, mask, workspace=ws)))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_other_streams_and_a_captured_graph():
    h, w, t, mask, up = problem(260, 2000, 128, 1, torch.bfloat16, 19)
    lab = t[:, 0]
    want = gbce.linear_ce_fwd_bwd_fused(h, w, lab)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [gbce.linear_ce_fwd_bwd_fused(h, w, lab, stream=s) for s in (s1, s2, s1, s2)]
    torch.cuda.synchronize()
    for out in outs:
        for a, b in zip(want[:3], out[:3]):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    hin = h.clone()
    with torch.cuda.graph(graph):
        out = gbce.linear_ce_fwd_bwd_fused(hin, w, lab)
    for k in range(3):
        hin.copy_(h if k != 1 else h * 0.5)
        graph.replay()
        again = gbce.linear_ce_fwd_bwd_fused(hin, w, lab)
        torch.cuda.synchronize()
        for a, b in zip(again[:3], out[:3]):
            assert torch.equal(a, b)


def test_gradient_against_differences():
    # fp32 at a smooth point: central differences of the fp64 loss
    h, w, t, mask, up = problem(6, 40, 8, 2, torch.float32, 21, margin=False, std=1.0)
    logp, state = gbce.linear_selective_logsoftmax(h, w, t, with_state=True)
    dh, dw = gbce.linear_selective_logsoftmax_bwd(h, w, t, up, logp, state)

    def loss(hh, ww):
        return (torch.log_softmax(hh @ ww.t(), 1).gather(1, t) * up.double()).sum()

    h64, w64 = h.double(), w.double()
    step = 1e-5
    for (x, d, f) in ((h64, dh, lambda y: loss(y, w64)), (w64, dw, lambda y: loss(h64, y))):
        for i, j in ((0, 0), (2, 5), (5, 7)):
            e = torch.zeros_like(x)
            e[i, j] = step
            num = (f(x + e) - f(x - e)) / (2 * step)
            # differences in fp64: 1e-10 from the step's square and the losses' rounding
            assert abs(float(num) - float(d[i, j])) <= 1e-5 * abs(float(num)) + 2e-8


def test_offsets_past_32_bits():
    # a table of more than 2^31 elements: its last rows count like its first
    V, D = 540000, 4096
    w = torch.zeros((V, D), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    hot = torch.tensor([0, 1, V // 2, V - 2, V - 1], device=DEV)
    w[hot] = torch.randn((5, D), generator=g, device=DEV).to(torch.bfloat16) * 0.05
    h = torch.randn((4, D), generator=g, device=DEV).to(torch.bfloat16)
    lab = torch.tensor([0, V - 1, V // 2, -100], device=DEV)
    out = gbce.linear_ce_fwd_bwd_fused(h, w, lab, reduction="sum")
    z = h[:3].double() @ w[hot].double().t()
    lse = torch.logsumexp(torch.cat([z, torch.full((3, 1), math.log(V - 5.0), device=DEV)], 1), 1)
    zt = z[torch.arange(3), torch.tensor([0, 4, 2])]
    assert abs(float(out.loss) - float((lse - zt).sum())) <= 1e-4
    p = torch.exp(z - lse[:, None])
    p[torch.arange(3), torch.tensor([0, 4, 2])] -= 1
    want = p.t() @ h[:3].double()
    got = out.dweight[hot].double()
    assert (got - want).norm() <= 2.0 ** -7 * want.norm()


def test_kernels_are_launched_and_counted():
    h, w, t, mask, up = problem(16, 64, 16, 1, torch.bfloat16, 23)
    n = gbce.kernel_launches()
    gbce.linear_ce_fwd_bwd_fused(h, w, t[:, 0])
    assert gbce.kernel_launches() > n + 4
    np.testing.assert_equal(tuple(t.shape), (16, 1))
