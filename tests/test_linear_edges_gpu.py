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
