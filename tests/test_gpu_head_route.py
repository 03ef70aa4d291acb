"""The router of the feature head (gs_expert_route_fwd / _bwd) against its
64-bit form."""

import pytest
import torch

from head8_util import route_bwd_ref, route_ref
from head_util import DEV, TYPES, check, gen, randn, sliced
from tile_gaussian_splat_gb300 import binding as gs

pytestmark = pytest.mark.gpu

# (tokens, experts, topk)
SHAPES = [(1, 1, 1), (1, 8, 2), (3, 2, 2), (5, 7, 3), (9, 16, 4), (64, 33, 8), (130, 64, 6),
          (33, 100, 17), (21, 256, 64), (12, 515, 64), (7, 1024, 33), (400, 4, 1), (2000, 20, 5),
          (257, 12, 12), (3001, 32, 32), (17, 130, 64), (40, 9, 4),
          (50, 31, 4), (50, 31, 5), (60, 63, 8), (60, 64, 16), (60, 64, 17), (33, 128, 16),
          (33, 127, 9), (30, 256, 32), (30, 250, 33), (20, 512, 9), (500, 8, 8), (70, 16, 16)]


def _check_fwd(logits, topk, keep=None, renormalise=True):
    ids, weights, counts, loss = gs.gs_expert_route_fwd(logits, topk, keep=keep,
                                                        renormalise=renormalise)
    r_ids, r_w, s_w, r_counts, r_loss, s_loss = route_ref(logits, topk, keep, renormalise)
    assert torch.equal(ids, r_ids)
    check(weights, r_w, s_w, "weights")
    assert torch.equal(counts, r_counts)
    assert abs(float(loss) - r_loss) <= s_loss + 2.0 ** -24 * r_loss
    return ids, weights, counts, loss


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("tokens,experts,topk", SHAPES)
def test_forward_and_backward(tokens, experts, topk, dtype):
    for n, (pad, renormalise, dropped) in enumerate([(0, True, 0.0), (3, False, 0.3),
                                                     (8, True, 0.3)]):
        g = gen(1000 * tokens + 10 * experts + topk + n)
        logits = sliced(2 * randn(g, tokens, experts, dtype=dtype), pad)
        keep = torch.rand(tokens, generator=g, device=DEV) >= dropped if dropped else None
        ids, weights, counts, loss = _check_fwd(logits, topk, keep, renormalise)
        gw = randn(g, tokens, topk)
        gl = randn(g, 1)
        wide = torch.full((tokens, experts + pad), 3.0, dtype=dtype, device=DEV)
        grad = gs.gs_expert_route_bwd(logits, ids, counts, gw, gl, renormalise=renormalise,
                                      out=wide[:, pad:])
        ref, slack = route_bwd_ref(logits, ids, counts, gw, gl, renormalise)
        check(grad, ref, slack, "grad_logits")
        assert bool((wide[:, :pad] == 3).all())
        for a, b in ((gw, None), (None, gl), (None, None)):
            grad = gs.gs_expert_route_bwd(logits, ids, counts, a, b, renormalise=renormalise)
            ref, slack = route_bwd_ref(logits, ids, counts, a, b, renormalise)
            check(grad, ref, slack, "grad_logits of one")


def test_without_the_balance_the_same_choice():
    g = gen(5)
    logits = randn(g, 999, 24)
    a = gs.gs_expert_route_fwd(logits, 3)
    b = gs.gs_expert_route_fwd(logits, 3, balance=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and b[2] is None and b[3] is None


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_ties_go_to_the_lowest_expert(dtype):
    g = gen(6)
    logits = torch.randint(0, 3, (700, 48), generator=g, device=DEV).to(dtype)
    logits[1] = 0
    logits[2, ::2] = -0.0  # equal to 0
    logits[2, 1::2] = 0.0
    ids = _check_fwd(logits, 9)[0]
    assert ids[1].tolist() == list(range(9)) and ids[2].tolist() == list(range(9))


@pytest.mark.parametrize("experts", [6, 16, 64, 300])
def test_masked_logits(experts):
    """Minus infinity is not chosen, not even where nothing else is left; the
    type's lowest value is a number like any other."""
    g = gen(experts)
    inf = float("inf")
    logits = randn(g, 40, experts)
    logits[0] = -inf
    logits[1, 1:] = -inf
    logits[2, 2:] = -inf
    logits[3] = torch.finfo(torch.float32).min
    logits[4, 3:] = torch.finfo(torch.float32).min
    logits[5] = torch.finfo(torch.float32).max
    logits[6, ::2] = -inf
    for renormalise in (True, False):
        ids, weights, counts, loss = _check_fwd(logits, 4, renormalise=renormalise)
        assert ids[0].tolist() == [-1] * 4 and ids[1].tolist() == [0, -1, -1, -1]
        assert int(counts[experts]) == 39 and bool(torch.isfinite(weights).all())
        gw, gl = randn(g, 40, 4), randn(g, 1)
        grad = gs.gs_expert_route_bwd(logits, ids, counts, gw, gl, renormalise=renormalise)
        ref, slack = route_bwd_ref(logits, ids, counts, gw, gl, renormalise)
        check(grad, ref, slack, "grad_logits")
        assert not bool(grad[0].any())


@pytest.mark.parametrize("experts,dtype", [(8, torch.float32), (24, torch.bfloat16), (9, torch.float16)])
def test_what_is_kept_out_is_not_looked_at(experts, dtype):
    g = gen(8)
    logits = randn(g, 500, experts, dtype=dtype)
    keep = torch.rand(500, generator=g, device=DEV) > 0.5
    a = gs.gs_expert_route_fwd(logits, 2, keep=keep)
    logits[~keep] = float("nan")
    b = gs.gs_expert_route_fwd(logits, 2, keep=keep.to(torch.uint8))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    grad = gs.gs_expert_route_bwd(logits, a[0], a[2], randn(g, 500, 2), randn(g, 1))
    assert not bool(grad[~keep].any()) and bool(torch.isfinite(grad).all())
    none = gs.gs_expert_route_fwd(logits, 2, keep=torch.zeros_like(keep))
    assert bool((none[0] == -1).all()) and not bool(none[1].any())
    assert not bool(none[2].any()) and float(none[3]) == 0
    grad = gs.gs_expert_route_bwd(logits, none[0], none[2], randn(g, 500, 2), randn(g, 1))
    assert not bool(grad.any())


def test_nan_and_infinity_stay_in_their_row():
    g = gen(9)
    logits = randn(g, 60, 16)
    clean = gs.gs_expert_route_fwd(logits, 3)
    logits[4, 7] = float("nan")
    logits[9, 2] = float("inf")
    ids, weights, counts, loss = gs.gs_expert_route_fwd(logits, 3)
    others = [t for t in range(60) if t not in (4, 9)]
    assert torch.equal(ids[others], clean[0][others])
    assert torch.equal(weights[others], clean[1][others])
    # first in the order, and their rows' softmax is no number
    assert int(ids[4, 0]) == 7 and int(ids[9, 0]) == 2
    assert bool(torch.isnan(weights[4]).all()) and bool(torch.isnan(weights[9, 0]))
    assert bool(torch.isnan(loss).all()) and int(counts[:16].sum()) == 180
    gw = randn(g, 60, 3)
    grad = gs.gs_expert_route_bwd(logits, ids, counts, gw)
    assert bool(torch.isfinite(grad[others]).all()) and bool(torch.isnan(grad[4]).all())


@pytest.mark.parametrize("dtype,bits", [(torch.float32, -0x400000), (torch.float16, -0x200),
                                        (torch.bfloat16, -0x40)])
@pytest.mark.parametrize("experts", [8, 12, 33, 200])
def test_a_nan_comes_first_whatever_its_sign(experts, dtype, bits):
    logits = randn(gen(experts), 9, experts, dtype=dtype)
    raw = logits.view({4: torch.int32, 2: torch.int16}[dtype.itemsize])
    raw[2, 5] = bits  # a NaN with its sign bit set
    logits[3, 1] = float("inf")
    logits[3, 6], logits[3, 2] = float("nan"), float("nan")
    assert bool(torch.isnan(logits[2, 5]))
    ids = gs.gs_expert_route_fwd(logits, 3)[0]
    assert int(ids[2, 0]) == 5 and ids[3].tolist() == [2, 6, 1]


def test_no_tokens():
    logits = torch.empty((0, 8), device=DEV)
    ids, weights, counts, loss = gs.gs_expert_route_fwd(logits, 2)
    assert ids.shape == (0, 2) and not bool(counts.any()) and float(loss) == 0
    assert gs.gs_expert_route_bwd(logits, ids, counts, weights, loss).shape == (0, 8)


def test_ids_that_are_none_are_skipped():
    """An id outside the experts counts as -1; the same expert twice adds twice."""
    g = gen(10)
    logits = randn(g, 6, 12)
    ids = torch.tensor([[3, 40], [3, -7], [-1, 2], [5, 5], [0, 11], [99, 1]], dtype=torch.int32,
                       device=DEV)
    gw = randn(g, 6, 2)
    clean = torch.where((ids < 0) | (ids >= 12), -1, ids)
    for renormalise in (True, False):
        grad = gs.gs_expert_route_bwd(logits, ids, None, gw, renormalise=renormalise)
        ref, slack = route_bwd_ref(logits, clean, None, gw, None, renormalise)
        check(grad, ref, slack, "grad_logits")


def test_the_range_checking_build_reports_such_ids():
    g = gen(10)
    logits = randn(g, 6, 12)
    ids = torch.tensor([[3, 4], [3, -1], [-1, -1], [5, 6], [0, 11], [9, 1]], dtype=torch.int32,
                       device=DEV)
    with gs.library(gs.LIB_DEBUG_PATH):
        for bad, code in ((None, 0), (12, 9), (-2, 9)):
            st = gs.new_status(DEV)
            if bad is not None:
                ids[4, 1] = bad
            gs.gs_expert_route_bwd(logits, ids, None, randn(g, 6, 2), d_status=st)
            assert int(st.item()) == code


def test_gradient_against_differences():
    """Central differences of the forward along random directions that keep
    the choice: 2h = 2e-3, its cubic term h^2 and the forward's rounding (1e-6
    over 2h at most) below 2e-3 of |gradient| |direction|."""
    g = gen(11)
    # experts a whole step apart, so that the choice holds
    logits = torch.rand((50, 10), generator=g, device=DEV).argsort(1).float()
    gw, gl = randn(g, 50, 3), 50 * randn(g, 1)

    for renormalise in (True, False):
        ids, _, counts, _ = gs.gs_expert_route_fwd(logits, 3, renormalise=renormalise)
        grad = gs.gs_expert_route_bwd(logits, ids, counts, gw, gl, renormalise=renormalise)
        v = randn(g, 50, 10)
        h = 1e-3

        def at(x):
            i, w, _, l = gs.gs_expert_route_fwd(x, 3, renormalise=renormalise)
            assert torch.equal(i, ids)
            return float((w.double() * gw.double()).sum() + l.double() * gl.double())

        diff = (at(logits + h * v) - at(logits - h * v)) / (2 * h)
        want = float((grad.double() * v.double()).sum())
        assert abs(diff - want) <= 2e-3 * float(grad.norm() * v.norm())


@pytest.mark.parametrize("experts,topk", [(8, 2), (40, 4), (300, 12)])
def test_gradients_that_have_most_in_common(experts, topk):
    """Renormalised weights sum to one, so an offset of all their gradients
    drops out: 1000 beside differences of 1 costs the rounding of the
    differences (2^-24 of 1000 each) and not that of sums of 1000."""
    g = gen(experts)
    logits = randn(g, 200, experts)
    ids = gs.gs_expert_route_fwd(logits, topk)[0]
    gw = 1000 + randn(g, 200, topk)
    grad = gs.gs_expert_route_bwd(logits, ids, None, gw)
    ref, slack = route_bwd_ref(logits, ids, None, gw - gw[:, :1], None, True)
    check(grad, ref, slack, "grad_logits")


def test_many_tokens_repeat_and_other_streams():
    g = gen(12)
    logits = randn(g, 300001, 16)
    keep = torch.rand(300001, generator=g, device=DEV) > 0.1
    gw, gl = randn(g, 300001, 2), randn(g, 1)
    a = gs.gs_expert_route_fwd(logits, 2, keep=keep)
    ga = gs.gs_expert_route_bwd(logits, a[0], a[2], gw, gl)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = gs.gs_expert_route_fwd(logits, 2, keep=keep, stream=side)
    gb = gs.gs_expert_route_bwd(logits, b[0], b[2], gw, gl, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and torch.equal(ga, gb)
    p = torch.softmax(logits.double(), 1) * keep[:, None]
    pairs = torch.bincount(a[0][keep].reshape(-1).long(), minlength=16)
    assert torch.equal(a[2][:16], pairs.int()) and int(a[2][16]) == int(keep.sum())
    loss = 16 * (pairs / pairs.sum() * p.sum(0) / keep.sum()).sum()
    # a block sums a few hundred tokens one after the other, then the blocks
    assert abs(float(loss) - float(a[3])) <= 1e-5 * float(loss)


def test_captured_and_replayed():
    g = gen(13)
    logits = randn(g, 5000, 32)
    gw, gl = randn(g, 5000, 4), randn(g, 1)
    graph = torch.cuda.CUDAGraph()
    gs.gs_expert_route_fwd(logits, 4)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = gs.gs_expert_route_fwd(logits, 4)
        grad = gs.gs_expert_route_bwd(logits, out[0], out[2], gw, gl)
    for seed in (1, 2):
        logits.copy_(randn(gen(seed), 5000, 32))
        graph.replay()
        want = gs.gs_expert_route_fwd(logits, 4)
        assert all(torch.equal(x, y) for x, y in zip(out, want))
        assert torch.equal(grad, gs.gs_expert_route_bwd(logits, want[0], want[2], gw, gl))


def test_offsets_beyond_32_bits():
    T, E = 2 ** 21 + 3, 1027  # in a row distance of 1027: 2.15e9 elements
    wide = torch.zeros((T, E), dtype=torch.float16, device=DEV)
    logits = wide[:, 3:11]
    logits[-5:] = randn(gen(14), 5, 8, dtype=torch.float16)
    ids, weights, counts, loss = gs.gs_expert_route_fwd(logits, 2)
    r = route_ref(logits[-5:], 2, None, True)
    assert torch.equal(ids[-5:], r[0])
    check(weights[-5:], r[1], r[2], "weights")
    assert bool((ids[:-5] == torch.tensor([0, 1], device=DEV)).all())
    gw = randn(gen(15), T, 2)
    out = torch.full_like(wide, 3.0)
    grad = gs.gs_expert_route_bwd(logits, ids, None, gw, out=out[:, 3:11])
    ref, slack = route_bwd_ref(logits[-5:], ids[-5:], None, gw[-5:], None, True)
    check(grad[-5:], ref, slack, "grad_logits")
    assert bool((out[:, :3] == 3).all()) and bool((out[:, 11:] == 3).all())


def test_refusals():
    x = torch.zeros((4, 8), device=DEV)
    ids = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    counts = torch.zeros(9, dtype=torch.int32, device=DEV)
    one = torch.zeros(1, device=DEV)
    for bad in (lambda: gs.gs_expert_route_fwd(x.double(), 2),
                lambda: gs.gs_expert_route_fwd(x, 0), lambda: gs.gs_expert_route_fwd(x, 9),
                lambda: gs.gs_expert_route_fwd(x[0], 1), lambda: gs.gs_expert_route_fwd(x.cpu(), 1),
                lambda: gs.gs_expert_route_fwd(x.t(), 2),
                lambda: gs.gs_expert_route_fwd(x, 2, keep=torch.ones(3, dtype=torch.bool,
                                                                     device=DEV)),
                lambda: gs.gs_expert_route_fwd(x, 2, keep=torch.ones(4, device=DEV)),
                lambda: gs.gs_expert_route_bwd(x, ids.long(), counts),
                lambda: gs.gs_expert_route_bwd(x, ids[:3], counts),
                lambda: gs.gs_expert_route_bwd(x, ids, counts, ids),
                lambda: gs.gs_expert_route_bwd(x, ids, None, None, one),
                lambda: gs.gs_expert_route_bwd(x, ids, counts[:8], None, one),
                lambda: gs.gs_expert_route_bwd(x, ids, counts, None, x),
                lambda: gs.gs_expert_route_bwd(x, ids, counts, out=torch.zeros((4, 7), device=DEV))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(gs.GsError, match="INVALID_ARG"):
        gs.gs_expert_route_fwd(torch.zeros((1, 1025), device=DEV), 2)
    with pytest.raises(gs.GsError, match="INVALID_ARG"):
        gs.gs_expert_route_fwd(torch.zeros((1, 100), device=DEV), 65)
