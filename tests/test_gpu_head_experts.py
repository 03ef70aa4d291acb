"""Pairs sorted by expert, rows dispatched and combined, against numpy's
stable sort and the 64-bit sums."""

import numpy as np
import pytest
import torch

from head_util import DEV, TYPES, U32, check, gen, randn, routed, sliced, sort_ref
from tile_gaussian_splat_gb300 import binding as gs
from tile_gaussian_splat_gb300 import build

pytestmark = pytest.mark.gpu


def _sorted(ids, experts):
    got = gs.gs_expert_sort(ids, experts)
    for g, r, name in zip(got, sort_ref(ids, experts), ("offsets", "order", "slots")):
        assert np.array_equal(g.cpu().numpy(), r), name
    return got


@pytest.mark.parametrize("tokens,topk,experts", [
    (1, 1, 1), (1, 2, 8), (3, 2, 5), (33, 1, 2), (500, 3, 7), (1000, 64, 64), (1025, 4, 1024),
    (4096, 2, 16), (70001, 2, 33), (300007, 3, 100), (1 << 20, 1, 257), (921600, 2, 16)])
def test_sort(tokens, topk, experts):
    rng = np.random.default_rng(tokens + experts)
    # ids beyond both ends drop their pair
    ids = rng.integers(-1, experts + 1, (tokens, topk)).astype(np.int32)
    _sorted(torch.from_numpy(ids).to(DEV), experts)


@pytest.mark.parametrize("tokens", [1, 100, 5000, 200000])
def test_sort_one_expert_none_and_extremes(tokens):
    for fill in (0, 6, -1, 7, 2 ** 31 - 1, -2 ** 31):
        _sorted(torch.full((tokens, 2), fill, dtype=torch.int32, device=DEV), 7)
    runs = torch.arange(tokens, device=DEV, dtype=torch.int32).reshape(-1, 1) * 7 // tokens
    _sorted(runs.to(torch.int32).contiguous(), 7)


def test_sort_of_nothing():
    offsets, order, slots = gs.gs_expert_sort(torch.empty((0, 2), dtype=torch.int32, device=DEV),
                                              5)
    assert offsets.tolist() == [0] * 6 and order.numel() == 0 and slots.shape == (0, 2)
    x = torch.empty((0, 16), device=DEV)
    xs = gs.gs_expert_dispatch(x, slots, offsets)
    assert xs.shape == (0, 16)
    assert gs.gs_expert_combine(xs, slots).shape == (0, 16)


CASES = [(1, 2, 8, 256), (1, 1, 1, 1), (7, 3, 5, 3), (100, 2, 4, 131), (257, 4, 16, 64),
         (1000, 2, 8, 1024), (333, 1, 3, 515), (50, 64, 64, 24), (2000, 5, 12, 72), (64, 2, 4, 4096)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("tokens,topk,experts,ch", CASES)
def test_rows_there_and_back(tokens, topk, experts, ch, dtype):
    for pad, drop in ((0, 0.0), (3, 0.3)):
        g = gen(tokens + ch)
        ids, offsets, order, slots = routed(tokens + ch, tokens, topk, experts, drop)
        kept = int(offsets[-1])
        x = sliced(randn(g, tokens, ch, dtype=dtype), pad)
        xs = torch.full((tokens * topk, ch), 5.0, dtype=dtype, device=DEV)
        gs.gs_expert_dispatch(x, slots, offsets, out=xs)
        assert torch.equal(xs[:kept], x[(order[:kept] // topk).long()])
        assert not bool(xs[kept:].any())
        ys = randn(g, tokens * topk, ch, dtype=dtype)
        ys[kept:] = float("nan")  # rows of no pair are never read
        w = randn(g, tokens, topk)
        w[slots < 0] = float("nan")  # nor are the weights of dropped pairs
        taken = torch.where((slots >= 0)[..., None], ys[slots.clamp(min=0).long()].double(), 0.0)
        wd = torch.where(slots >= 0, w.double(), 0.0)[..., None]
        for weights, f in ((w, wd), (None, torch.ones_like(wd))):
            wide = torch.full((tokens, ch + pad), 3.0, dtype=dtype, device=DEV)
            y = gs.gs_expert_combine(ys, slots, weights, out=wide[:, pad:])
            check(y, (taken * f).sum(1), (topk + 2) * U32 * (taken * f).abs().sum(1), "y")
            assert bool((wide[:, :pad] == 3).all())
        gy = sliced(randn(g, tokens, ch, dtype=dtype), pad)
        gys, gw = gs.gs_expert_combine_bwd(gy, ys, slots, w, offsets)
        want = torch.zeros((tokens * topk, ch), dtype=torch.float64, device=DEV)
        want[slots[slots >= 0].long()] = (gy.double()[:, None] * wd)[slots >= 0]
        check(gys, want, 2 * U32 * want.abs(), "grad_ys")
        terms = taken * gy.double()[:, None]
        check(gw, terms.sum(2), (ch + 2) * U32 * terms.abs().sum(2), "grad_weights")
        plain, none = gs.gs_expert_combine_bwd(gy, ys, slots, None, offsets)
        assert none is None
        assert torch.equal(plain, gs.gs_expert_dispatch(gy, slots, offsets))


def test_a_token_without_a_pair_gives_zero():
    ids, offsets, order, slots = routed(3, 40, 2, 4, drop=1.0)
    ys = torch.full((80, 33), float("inf"), device=DEV)
    assert int(offsets[-1]) == 0
    assert not bool(gs.gs_expert_combine(ys, slots, torch.ones((40, 2), device=DEV)).any())
    gys, gw = gs.gs_expert_combine_bwd(torch.ones((40, 33), device=DEV), ys, slots,
                                       torch.ones((40, 2), device=DEV), offsets)
    assert not bool(gys.any()) and not bool(gw.any())


def test_offsets_beyond_32_bits():
    tokens, ch = 2 ** 20 + 3, 1030
    ids = torch.zeros((tokens, 2), dtype=torch.int32, device=DEV)
    ids[:, 1] = 1
    offsets, order, slots = gs.gs_expert_sort(ids, 2)
    x = torch.empty((tokens, ch), dtype=torch.float16, device=DEV)
    x[:] = (torch.arange(tokens, device=DEV) % 1001).to(torch.float16)[:, None]
    xs = gs.gs_expert_dispatch(x, slots, offsets)  # 2.16e9 elements
    assert torch.equal(xs[:tokens], x) and torch.equal(xs[tokens:], x)
    w = torch.full((tokens, 2), 0.5, device=DEV)
    w[:, 1] = 0.25
    assert torch.equal(gs.gs_expert_combine(xs, slots, w), x * 0.75)
    gys, gw = gs.gs_expert_combine_bwd(x, xs, slots, w, offsets)
    assert torch.equal(gys[tokens:], x * 0.25) and torch.equal(gys[:tokens], x * 0.5)
    want = ch * x[:, :1].double() ** 2
    check(gw, want.expand(-1, 2), (ch + 2) * U32 * want.expand(-1, 2), "grad_weights")


def test_gradient_against_differences():
    """The combine is linear in ys and in the weights, so a difference of any
    width is the gradient up to the forward's rounding (1e-7 of its terms)."""
    g = gen(5)
    ids, offsets, order, slots = routed(5, 60, 3, 6, 0.2)
    ys, w, gy = randn(g, 180, 40), randn(g, 60, 3), randn(g, 60, 40)
    gys, gw = gs.gs_expert_combine_bwd(gy, ys, slots, w, offsets)
    loss = lambda a, b: float((gs.gs_expert_combine(a, slots, b).double() * gy.double()).sum())
    for t, grad, up, down in ((ys, gys, lambda v: loss(ys + v, w), lambda v: loss(ys - v, w)),
                              (w, gw, lambda v: loss(ys, w + v), lambda v: loss(ys, w - v))):
        v = randn(g, *t.shape)
        want = float((grad.double() * v.double()).sum())
        assert abs((up(v) - down(v)) / 2 - want) <= 1e-5 * float(grad.norm() * v.norm())


def test_repeatability_and_another_stream():
    g = gen(6)
    ids, _, _, _ = routed(6, 30000, 2, 8, 0.1)
    side = torch.cuda.Stream()
    x, gy, w = randn(g, 30000, 96), randn(g, 30000, 96), randn(g, 30000, 2)

    def passes(stream):
        offsets, order, slots = gs.gs_expert_sort(ids, 8, stream=stream)
        xs = gs.gs_expert_dispatch(x, slots, offsets, stream=stream)
        y = gs.gs_expert_combine(xs, slots, w, stream=stream)
        return (offsets, order, slots, xs, y,
                *gs.gs_expert_combine_bwd(gy, xs, slots, w, offsets, stream=stream))

    first = passes(None)
    side.wait_stream(torch.cuda.current_stream())
    second = passes(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, second))


def test_indices_outside_their_arrays_are_skipped_and_reported():
    build.build()
    ids, offsets, order, slots = routed(8, 100, 2, 4, 0.0)
    x = torch.ones((100, 48), device=DEV)
    bad_slots, bad_offsets = slots.clone(), offsets.clone()
    bad_slots[7, 1] = 200
    bad_offsets[-1] = 10 ** 6
    for lib, code in ((gs.LIB_PATH, 0), (gs.LIB_DEBUG_PATH, 9)):
        with gs.library(lib):
            st = gs.new_status(DEV)
            xs = gs.gs_expert_dispatch(x, slots, offsets, d_status=st)
            gs.check_status(st)
            st = gs.new_status(DEV)
            y = gs.gs_expert_combine(xs, bad_slots, d_status=st)
            assert int(st.item()) == code
            assert bool((y[7] == 1).all()) and bool((y[:7] == 2).all())
            for call in (lambda st: gs.gs_expert_dispatch(x, bad_slots, offsets, d_status=st),
                         lambda st: gs.gs_expert_dispatch(x, slots, bad_offsets, d_status=st),
                         lambda st: gs.gs_expert_combine_bwd(x, xs, bad_slots, None, offsets,
                                                             d_status=st)):
                st = gs.new_status(DEV)
                call(st)
                assert int(st.item()) == code


def test_refusals():
    x = torch.zeros((4, 8), device=DEV)
    ids = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    offsets, order, slots = gs.gs_expert_sort(ids, 3)
    xs = gs.gs_expert_dispatch(x, slots, offsets)
    w = torch.ones((4, 2), device=DEV)
    for bad in (lambda: gs.gs_expert_sort(ids.long(), 3), lambda: gs.gs_expert_sort(ids[0], 3),
                lambda: gs.gs_expert_sort(ids.t(), 3),
                lambda: gs.gs_expert_dispatch(x[:3], slots, offsets),
                lambda: gs.gs_expert_dispatch(x.int(), slots, offsets),
                lambda: gs.gs_expert_dispatch(x, slots, offsets.long()),
                lambda: gs.gs_expert_combine(xs[:7], slots),
                lambda: gs.gs_expert_combine(xs, slots, w.half()),
                lambda: gs.gs_expert_combine(xs, slots, w[:3]),
                lambda: gs.gs_expert_combine_bwd(x.half(), xs, slots, w, offsets),
                lambda: gs.gs_expert_combine(xs.cpu(), slots)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: gs.gs_expert_sort(ids, 0), lambda: gs.gs_expert_sort(ids, 1025),
                lambda: gs.gs_expert_sort(torch.zeros((1, 65), dtype=torch.int32, device=DEV), 3)):
        with pytest.raises((gs.GsError, RuntimeError)):
            bad()
