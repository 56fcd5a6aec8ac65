"""Edges of the linear calls and the table's lookup: tiles whose last rows end
inside a warp, upstream sums that cancel, long runs of one token, outputs that
are parts of other tensors."""

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


def draw(rows, V, D, K, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = (torch.randn((V, D), generator=g, device=DEV) * (2.0 / D ** 0.5)).to(dtype)
    h = torch.randn((rows, D), generator=g, device=DEV).to(dtype)
    t = torch.randint(0, V, (rows, K), generator=g, device=DEV)
    up = torch.randn((rows, K), generator=g, device=DEV) / rows
    return h, w, t, up


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,V,D", [
    (1, 33, 72), (31, 65, 136), (33, 97, 200), (97, 191, 264), (159, 1057, 520),  # single CTAs' tiles
    (1090, 20003, 520),                                                           # pairs' tiles
])
def test_gradients_of_tiles_that_end_inside_a_warp(rows, V, D, dtype):
    # of a tile's last 32 rows (dhidden) or columns of logits (dweight) some
    # lanes of a warp have one and the others none, over several blocks of 32
    # columns of the output
    T = 0.9
    h, w, t, up = draw(rows, V, D, 1, dtype, rows + V)
    logp, state = gbce.linear_selective_logsoftmax(h, w, t, T, with_state=True)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    start = torch.randn((V, D), device=DEV).to(dtype)
    dh, dw = gbce.linear_selective_logsoftmax_bwd(h, w, t, up, logp, state, T, dev_status=st)
    acc = start.clone()
    gbce.linear_selective_logsoftmax_bwd(h, w, t, up, logp, state, T, dweight=acc, accumulate=True,
                                         want_dhidden=False, dev_status=st)
    assert int(st) == 0
    live = torch.ones(rows, dtype=torch.bool, device=DEV)
    p, lp, comp, ez = ref.rows_of(h, w, t, T, live)
    ref.assert_within(logp, lp, ref.logp_bound(lp, comp, ez), "log p")
    dz, size = ref.selective_dz(p, lp, comp, t, up.double(), T)
    rdh, rdw, bh, bw = ref.products(dz, size, h.double(), w.double(), ez, dtype)
    ref.assert_within(dh, rdh, bh, "dhidden")
    ref.assert_within(dw, rdw, bw, "dweight")
    both = start.double() + rdw
    # the sum's addition and rounding on top
    ref.assert_within(acc, both, bw + (ref.HALF[dtype] + ref.U) * both.abs(), "dweight +=")


def elapsed(call, n=10):
    for _ in range(3):
        call()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    a.record()
    for _ in range(n):
        call()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / n


def test_lookup_gradient_takes_no_longer_for_one_token_than_for_many():
    # 2 rows >= vocab: the zeros of a fresh table are written by CTAs that find
    # out which of their rows are named.  Walking the run of a token that every
    # row names cost one of them 8192 loads in a row (ten times the call).
    rows, V, D = 262144, 400000, 8
    g = torch.Generator(device=DEV).manual_seed(2)
    go = torch.randn((rows, D), generator=g, device=DEV)
    spread = torch.randint(0, V, (rows,), generator=g, device=DEV)
    one = torch.full((rows,), 5, device=DEV)
    t = [elapsed(lambda: gbce.embedding_lookup_bwd(go, tok, V)) for tok in (spread, one)]
    assert t[1] <= 3.0 * t[0], t


@pytest.mark.parametrize("rows,V", [(64, 100), (700, 47), (4000, 600), (9000, 33), (30000, 17)])
def test_rows_beside_long_runs_get_their_zeros(rows, V):
    # runs of one token from 1 to all the rows, on every place of a block of 16
    # table rows, among neighbours that nobody names and that somebody does
    go = torch.ones((rows, 3), device=DEV)
    for at in range(min(V, 17)):
        for other in (at, (at + 1) % V, (at + 5) % V, V - 1):
            for n in (1, 31, 33, rows - 2):
                tok = torch.full((rows,), at, device=DEV)
                tok[:max(0, rows - 1 - n)] = -100
                tok[rows // 2] = other
                d = gbce.embedding_lookup_bwd(go, tok, V, dtable=torch.full((V, 3), 7.0, device=DEV))
                want = torch.bincount(tok[tok >= 0], minlength=V).float()  # whole numbers: exact
                assert torch.equal(d, want[:, None].expand(V, 3)), (at, other, n)


@pytest.mark.parametrize("rows,V,D", [(256, 3, 8), (300, 40, 64)])
def test_upstream_sums_that_cancel(rows, V, D):
    # K = 16: indices 8..15 repeat 0..7 with each upstream negated to within
    # 1e-4, so that every column's summed upstream (and every element of the
    # gradients) is a sum of terms about 1 that cancels to about 1e-4.
    #
    # A gathered column's dz is g_t (1 - p_t) / T - g_o p_t / T with g_t and g_o
    # the exact sums.  Sums of 16 fp32 values in fp64 and their one rounding are
    # within 2 u of them; 1 - p_t and p_t come from the saved log p, off by
    # comp (2 ez + 2 u (|log p| + 64)) + 4 u |log p| at most, which relative to
    # either is at most 2 ez + 2 u (|log p| + 64) + 4 u (|log p| + 1) (for |log
    # p| p <= 1 - p); expm1, exp, two products and the sum 8 u; the other
    # columns 2 ez + 16 u of |G| p_j / T.  Sums in fp32 are off by up to 16 u
    # of the terms, a thousand times as much of what is left.
    T, K = 0.8, 16
    h, w, t, _ = draw(rows, V, D, K, torch.float32, rows)
    g = torch.Generator(device=DEV).manual_seed(92)
    up = torch.randn((rows, K), generator=g, device=DEV)
    t[:, 8:] = t[:, :8]
    up[:, 8:] = -up[:, :8] + 1e-4 * torch.randn((rows, 8), generator=g, device=DEV)
    logp, state = gbce.linear_selective_logsoftmax(h, w, t, T, with_state=True)
    dh, dw = gbce.linear_selective_logsoftmax_bwd(h, w, t, up, logp, state, T)

    live = torch.ones(rows, dtype=torch.bool, device=DEV)
    p, lp, comp, ez = ref.rows_of(h, w, t, T, live)
    u64 = up.double()
    total = u64.sum(1, keepdim=True)
    dz, off = -total * p, total.abs() * p * (2 * ez + 16 * ref.U)
    for k in range(K):
        own = t[:, k:k + 1]
        mine = torch.where(t == own, u64, 0.0).sum(1, keepdim=True)
        other = torch.where(t == own, 0.0, u64).sum(1, keepdim=True)
        pt, ct, size = p.gather(1, own), comp[:, k:k + 1], lp[:, k:k + 1].abs()
        rel = 2 * ez + 2 * ref.U * (size + 64) + 4 * ref.U * (size + 1) + 10 * ref.U
        dz.scatter_(1, own, mine * ct - other * pt)
        off.scatter_(1, own, (mine.abs() * ct + other.abs() * pt) * rel)
    dz, off = dz / T, off / T + 4 * ref.U * dz.abs() / T  # and what three bf16 planes leave
    for got, want, size, err, n, what in (
            (dh, dz @ w.double(), dz.abs() @ w.double().abs(), off @ w.double().abs(), V, "dhidden"),
            (dw, dz.t() @ h.double(), dz.abs().t() @ h.double().abs(), off.t() @ h.double().abs(), rows, "dweight")):
        ref.assert_within(got, want, 1.01 * err + (n / 8 + 16) * ref.U * size + ref.U * want.abs(), what)


def test_gradients_without_rows():
    w = torch.randn((300, 64), device=DEV, dtype=torch.bfloat16)
    h = torch.empty((0, 64), device=DEV, dtype=torch.bfloat16)
    lab = torch.empty((0,), device=DEV, dtype=torch.int64)
    logp, state = torch.empty((0,), device=DEV), torch.empty((0, 2), device=DEV)
    calls = [lambda **kw: gbce.linear_ce_fwd_bwd_fused(h, w, lab, **kw)[1:3],
             lambda **kw: gbce.linear_ce_bwd(h, w, lab, 1.0, logp, state, torch.zeros((), dtype=torch.int64), **kw),
             lambda **kw: gbce.linear_selective_logsoftmax_bwd(h, w, lab, logp, logp, state, **kw)]
    for call in calls:
        before = w.clone()
        with pytest.raises(gbce.GbceError):
            call(dweight=w)
        with pytest.raises(gbce.GbceError):
            call(want_dhidden=False, want_dweight=False)
        assert torch.equal(w, before)
        dh, dw = call(want_dweight=False)
        assert dh.shape == (0, 64) and dw is None
        dh, dw = call(want_dhidden=False, dweight=torch.full_like(w, 7.0))
        assert dh is None and not dw.any()
        wide = torch.full((300, 70), 7.0, device=DEV, dtype=torch.bfloat16)
        dh, dw = call(dweight=wide[:, :64])
        assert dh.shape == (0, 64) and not dw.any() and (wide[:, 64:] == 7.0).all()
        dh, dw = call(dweight=torch.full_like(w, 7.0), accumulate=True)
        assert (dw == 7.0).all()


def test_lookup_of_a_scalar_token_into_a_part_of_another_tensor():
    # one row of `dim` elements: its own unit stride counts, like any row's
    table = torch.randn((10, 16), device=DEV)
    buf = torch.full((64,), 7.0, device=DEV)
    with pytest.raises(ValueError, match="unit stride"):
        gbce.embedding_lookup(table, torch.tensor(3), out=buf[0:32:2])
    assert (buf == 7.0).all()
    out = gbce.embedding_lookup(table, torch.tensor(3), out=buf[5:21])
    assert torch.equal(out, table[3]) and (buf[:5] == 7.0).all() and (buf[21:] == 7.0).all()
    one = torch.randn((4, 1), device=DEV)
    out = gbce.embedding_lookup(one, torch.tensor(2), out=buf[0:64:64])
    assert torch.equal(out, one[2]) and (buf[22:] == 7.0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradient_of_a_scalar_tokens_lookup(dtype):
    # tokens of any shape have rows of shape [*tokens.shape, dim], [dim] for a scalar
    table = torch.randn((10, 16), device=DEV).to(dtype)
    tok = torch.tensor(3, device=DEV)
    row = gbce.embedding_lookup(table, tok, 2.0)
    d = gbce.embedding_lookup_bwd(row, tok, 10, 2.0)
    want = torch.zeros_like(table)
    want[3] = 2.0 * row  # a power of two: exact
    assert torch.equal(d, want)
    acc = gbce.embedding_lookup_bwd(row, tok, 10, 2.0, dtable=d, accumulate=True)
    assert acc is d and torch.equal(d, 2.0 * want)
    with pytest.raises(ValueError, match="unit stride"):
        gbce.embedding_lookup_bwd(torch.zeros(32, device=DEV, dtype=dtype)[::2], tok, 10)
    with pytest.raises(ValueError, match="shape"):
        gbce.embedding_lookup_bwd(row, tok[None], 10)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V,K", [(1, 1), (2, 2), (3, 5), (16, 16)])
def test_nan_where_every_column_is_gathered(V, K, dtype):
    # no column is left for the tiles' sums, so the NaN is in gathered logits alone
    nan = float("nan")
    g = torch.Generator(device=DEV).manual_seed(V)
    h = torch.randn((3, 8), generator=g, device=DEV).to(dtype)
    w = torch.randn((V, 8), generator=g, device=DEV).to(dtype)
    t = (torch.arange(K, device=DEV) % V).expand(3, K).contiguous()
    clean, cstate = gbce.linear_selective_logsoftmax(h, w, t, with_state=True)
    assert torch.isfinite(clean).all()
    hn = h.clone()
    hn[1] = nan  # a NaN row: its log-probs, its state and its gradients, nobody else's
    logp, state = gbce.linear_selective_logsoftmax(hn, w, t, with_state=True)
    assert torch.isnan(logp[1]).all() and torch.isnan(state[1, 1])
    assert torch.equal(logp[[0, 2]], clean[[0, 2]]) and torch.equal(state[[0, 2]], cstate[[0, 2]])
    dh, _ = gbce.linear_selective_logsoftmax_bwd(hn, w, t, torch.ones_like(logp), logp, state)
    assert torch.isnan(dh[1]).all() and torch.isfinite(dh[[0, 2]]).all()
    out = gbce.linear_ce_fwd_bwd_fused(hn, w, t[:, 0], reduction="none", want_logp=True)
    assert torch.isnan(out.loss[1]) and torch.isnan(out.logp[1]) and torch.isfinite(out.loss[[0, 2]]).all()
    wn = w.clone()
    wn[V - 1] = nan  # a NaN column: every row has it among its others
    logp, state = gbce.linear_selective_logsoftmax(h, wn, t, with_state=True)
    assert torch.isnan(logp).all() and torch.isnan(state[:, 1]).all()


def graph_of(call, n=10):
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(n):
            call()
    return graph


def test_fewer_targets_take_no_longer_than_more():
    # six CTAs make the logits of 300 x 128: with the 1200 gathered ones of four
    # targets left to their warps a call took over twice as long as with 16
    # targets, whose logits the packing makes
    h, w, t, _ = draw(300, 128, 4096, 16, torch.bfloat16, 5)
    four = t[:, :4].contiguous()
    ms = [elapsed(graph_of(lambda: gbce.linear_selective_logsoftmax(h, w, x)).replay) for x in (four, t)]
    assert ms[0] <= 1.5 * ms[1], ms


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,V,D,K", [(1000, 64, 200, 1), (600, 130, 72, 2), (129, 65, 264, 4), (200, 40, 64, 6)])
def test_many_rows_of_few_columns(rows, V, D, K, dtype):
    h, w, t, _ = draw(rows, V, D, K, dtype, rows)
    logp, state = gbce.linear_selective_logsoftmax(h, w, t, 0.8, with_state=True)
    live = torch.ones(rows, dtype=torch.bool, device=DEV)
    p, lp, comp, ez = ref.rows_of(h, w, t, 0.8, live)
    ref.assert_within(logp, lp, ref.logp_bound(lp, comp, ez), "log p")
    lab = t[:, 0].contiguous()
    both = gbce.linear_ce_fwd_bwd_fused(h, w, lab, want_logp=True)
    f = gbce.linear_ce_fwd(h, w, lab)
    assert torch.equal(both.logp, f.logp) and torch.equal(both.loss, f.loss)
