"""embedding_lookup and its gradient against the definition in 64 bits, and
the tied table's whole training step."""

import math

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


def tokens_of(kind, rows, V, g):
    if kind == "one":            # every row names the same token
        t = torch.full((rows,), V - 1, device=DEV)
    elif kind == "common":       # as in text: a few very common ones
        u = torch.rand(rows, generator=g, device=DEV, dtype=torch.float64)
        t = torch.exp(u * math.log(V + 1.0)).long().sub_(1).clamp_(0, V - 1)
    else:
        t = torch.randint(0, V, (rows,), generator=g, device=DEV)
    if rows > 4 and kind != "one":
        t[rows // 3] = -100
        t[-1] = -100
    return t


def grad_ref(g, t, V, scale):
    """The sum and the sum of magnitudes per table row, in fp64."""
    live = t != -100
    s = torch.zeros((V, g.shape[1]), dtype=torch.float64, device=DEV)
    a = torch.zeros_like(s)
    s.index_add_(0, t[live], g[live].double() * scale)
    a.index_add_(0, t[live], g[live].double().abs() * abs(scale))
    n = torch.zeros(V, dtype=torch.float64, device=DEV).index_add_(
        0, t[live], torch.ones(int(live.sum()), dtype=torch.float64, device=DEV))
    return s, a, n[:, None]


SIZES = [(1, 1, 1), (1, 7, 8), (5, 3, 7), (33, 10, 64), (64, 1000, 129), (257, 40, 72),
         (1000, 151, 256), (4099, 30011, 40), (9000, 33, 24), (20000, 70000, 16)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,V,D", SIZES)
@pytest.mark.parametrize("kind", ["uniform", "common", "one"])
def test_lookup_and_gradient(rows, V, D, dtype, kind):
    g = torch.Generator(device=DEV).manual_seed(rows + V)
    table = torch.randn((V, D), generator=g, device=DEV).to(dtype)
    t = tokens_of(kind, rows, V, g)
    scale = 1.7
    out = gbce.embedding_lookup(table, t, scale)
    live = (t != -100)[:, None]
    # one fp32 product of an fp32 scale, then the type's rounding
    want = torch.where(live, table[t.clamp(min=0)].float() * torch.tensor(scale, device=DEV),
                       torch.zeros((), device=DEV)).to(dtype)
    assert torch.equal(out, want)
    go = torch.randn((rows, D), generator=g, device=DEV).to(dtype)
    go[t == -100] = math.nan  # what padding rows hold does not matter
    s, a, n = grad_ref(torch.nan_to_num(go), t, V, scale)
    got = gbce.embedding_lookup_bwd(go, t, V, scale)
    # n fp32 additions and the scale's product, then the type's rounding
    bound = (n + 3) * ref.U * a + ref.HALF[dtype] * s.abs() * 1.001
    ref.assert_within(got, s, bound, "dtable")
    start = torch.randn((V, D), generator=g, device=DEV).to(dtype)
    acc = start.clone()
    gbce.embedding_lookup_bwd(go, t, V, scale, dtable=acc, accumulate=True)
    sum_ = start.double() + s
    ref.assert_within(acc, sum_, (n + 3) * ref.U * (a + start.double().abs())
                      + ref.HALF[dtype] * sum_.abs() * 1.001, "dtable +=")
    assert torch.equal(acc[n[:, 0] == 0], start[n[:, 0] == 0])
    again = gbce.embedding_lookup_bwd(go, t, V, scale)
    assert torch.equal(again, got)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (8, 8), (5, 3)])
def test_strided_and_misaligned(dtype, pad, shift):
    g = torch.Generator(device=DEV).manual_seed(3)
    V, D, rows = 60, 40, 300

    def wide(t):
        buf = torch.full((t.shape[0] * (D + pad) + shift,), math.nan, dtype=dtype, device=DEV)
        view = buf[shift:].view(t.shape[0], D + pad)[:, :D]
        view.copy_(t)
        return view

    table = torch.randn((V, D), generator=g, device=DEV).to(dtype)
    go = torch.randn((rows, D), generator=g, device=DEV).to(dtype)
    t = tokens_of("uniform", rows, V, g)
    out = gbce.embedding_lookup(wide(table), t, 0.5, out=wide(go))
    assert torch.equal(out, gbce.embedding_lookup(table, t, 0.5))
    d = gbce.embedding_lookup_bwd(wide(go), t, V, 0.5, dtable=wide(table))
    assert torch.equal(d, gbce.embedding_lookup_bwd(go, t, V, 0.5))
    for x in (out, d):
        if pad:
            gap = torch.as_strided(x, (x.shape[0] - 1, pad), (x.stride(0), 1), x.storage_offset() + D)
            assert torch.isnan(gap).all()


def test_bad_tokens_empty_calls_and_shapes():
    table = torch.randn((10, 16), device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    t = torch.tensor([[1, 10, -100], [-5, 1 << 40, 9]], device=DEV)
    out = gbce.embedding_lookup(table, t, dev_status=st)
    assert out.shape == (2, 3, 16) and int(st) == gbce.DEV_BAD_INDEX
    bad = torch.tensor([[False, True, False], [True, True, False]], device=DEV)
    assert torch.isnan(out[bad]).all() and not out[0, 2].any()
    assert torch.equal(out[1, 2], table[9])
    st.zero_()
    d = gbce.embedding_lookup_bwd(torch.ones((2, 3, 16), device=DEV), t, 10, dev_status=st)
    assert int(st) == gbce.DEV_BAD_INDEX
    assert (d[[1, 9]] == 1).all() and float(d.sum()) == 32.0
    none = gbce.embedding_lookup_bwd(torch.ones((0, 16), device=DEV), t.view(-1)[:0], 10,
                                     dtable=torch.full((10, 16), 7.0, device=DEV))
    assert not none.any()
    keep = torch.full((10, 16), 7.0, device=DEV)
    gbce.embedding_lookup_bwd(torch.ones((0, 16), device=DEV), t.view(-1)[:0], 10, dtable=keep,
                              accumulate=True)
    assert (keep == 7.0).all()
    assert gbce.embedding_lookup(table, t[:0]).shape == (0, 3, 16)
    assert gbce.embedding_lookup(table, torch.tensor(3)).shape == (16,)
    # an ignored token may be one that the table has
    z = gbce.embedding_lookup(table, torch.tensor([3, 4]), ignore_index=3)
    assert not z[0].any() and torch.equal(z[1], table[4])


def test_offsets_past_32_bits():
    V, D = 540000, 4096
    table = torch.zeros((V, D), dtype=torch.bfloat16, device=DEV)
    t = torch.tensor([0, V - 1, V // 2, V - 1, -100], device=DEV)
    table[V - 1] = 3.0
    out = gbce.embedding_lookup(table, t, 0.5)
    assert (out[[1, 3]] == 1.5).all() and not out[[0, 2, 4]].any()
    d = gbce.embedding_lookup_bwd(torch.ones((5, D), dtype=torch.bfloat16, device=DEV), t, V, 2.0,
                                  dtable=table.fill_(7.0))
    assert (d[V - 1] == 4.0).all() and (d[0] == 2.0).all() and (d[V // 2] == 2.0).all()
    assert float(d.sum(dtype=torch.float64)) == 8.0 * D


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V,D", [(1000, 31), (1003, 7), (999, 130), (17, 1), (5, 3)])
def test_zeros_reach_every_element_of_odd_tables(dtype, V, D):
    for shift in (0, 1):
        buf = torch.full((V * D + shift + 1,), 7.0, dtype=dtype, device=DEV)
        d = buf[shift:shift + V * D].view(V, D)
        gbce.embedding_lookup_bwd(torch.ones((1, D), dtype=dtype, device=DEV),
                                  torch.tensor([V // 2], device=DEV), V, dtable=d)
        assert float(d.double().sum()) == D and (d[V // 2] == 1).all()
        assert float(buf[-1]) == 7.0 and (shift == 0 or float(buf[0]) == 7.0)


def test_streams_and_a_captured_graph():
    g = torch.Generator(device=DEV).manual_seed(8)
    t = tokens_of("common", 5000, 2000, g)
    go = torch.randn((5000, 72), generator=g, device=DEV)
    want = gbce.embedding_lookup_bwd(go, t, 2000)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [gbce.embedding_lookup_bwd(go, t, 2000, stream=s) for s in (s1, s2, s1)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    tin = t.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gbce.embedding_lookup_bwd(go, tin, 2000)
    for k in range(2):
        tin.copy_(t.roll(k))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, gbce.embedding_lookup_bwd(go, t.roll(k), 2000))


def test_workspace_may_hold_anything():
    g = torch.Generator(device=DEV).manual_seed(9)
    t = tokens_of("common", 3000, 500, g)
    go = torch.randn((3000, 40), generator=g, device=DEV)
    n = int(gbce.load_library().gbce_embedding_workspace_size(3000, 500, 40))
    outs = [gbce.embedding_lookup_bwd(go, t, 500, workspace=torch.full((n,), f, dtype=torch.uint8,
                                                                       device=DEV)) for f in (0, 255)]
    assert torch.equal(*outs)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_tied_tables_training_step(dtype):
    # tokens -> table rows -> hidden states -> loss; the head's gradient of the
    # table and the lookup's meet in one buffer
    g = torch.Generator(device=DEV).manual_seed(10)
    rows, V, D = 300, 900, 64
    scale = math.sqrt(D)
    table = (torch.randn((V, D), generator=g, device=DEV) * 0.3).to(dtype)
    tok = tokens_of("common", rows, V, g)
    lab = tok.roll(-1)
    x = gbce.embedding_lookup(table, tok, scale)
    r = gbce.linear_ce_fwd_bwd_fused(x, table, lab)
    head = r.dweight.clone()
    total = gbce.embedding_lookup_bwd(r.dhidden, tok, V, scale, dtable=r.dweight, accumulate=True)
    assert total is r.dweight
    s, a, n = grad_ref(torch.nan_to_num(r.dhidden), tok, V, scale)
    want = head.double() + s
    ref.assert_within(total, want, (n + 3) * ref.U * (a + head.double().abs())
                      + ref.HALF[dtype] * want.abs() * 1.001, "tied gradient")
    # and against autograd in 64 bits
    t64 = table.double().requires_grad_()
    live = (tok != -100)[:, None]
    h64 = torch.where(live, t64[tok.clamp(min=0)] * scale, torch.zeros((), dtype=torch.float64, device=DEV))
    loss = torch.nn.functional.cross_entropy(h64 @ t64.t(), lab, ignore_index=-100)
    loss.backward()
    tol = 6 * ref.HALF[dtype] if dtype == torch.bfloat16 else 2e-5  # x, dz, dhidden, two sums, total
    assert abs(float(r.loss) - float(loss)) <= (2e-2 if dtype == torch.bfloat16 else 1e-5) * float(loss)
    assert (total.double() - t64.grad).norm() <= tol * t64.grad.norm()
