"""The experts' products and their gradients against the 64-bit form."""

import pytest
import torch

from head_util import (DEV, TYPES, check, gen, linear_bwd_ref, linear_ref, randn, routed)
from tile_gaussian_splat_gb300 import binding as gs
from tile_gaussian_splat_gb300 import build

pytestmark = pytest.mark.gpu

# tokens, topk, experts, in, out, experts that get rows
SHAPES = [
    (1, 2, 8, 256, 1024, None), (1, 1, 1, 1, 1, None), (2, 2, 3, 8, 8, None),
    (3, 1, 4, 17, 5, None), (40, 2, 4, 64, 128, None), (129, 1, 1, 72, 256, None),
    (128, 1, 2, 64, 64, [1]), (127, 2, 5, 131, 259, None), (300, 3, 6, 264, 72, [0, 3, 5]),
    (700, 2, 4, 512, 384, None), (1000, 2, 16, 128, 520, None), (2500, 2, 3, 200, 136, None),
    (900, 1, 64, 96, 48, None), (4000, 2, 2, 256, 256, [1]), (60, 2, 1024, 24, 16, None),
    (1500, 2, 4, 1032, 40, None), (513, 1, 1, 33, 513, None),
    (10000, 2, 3, 136, 520, None), (9000, 2, 5, 512, 384, None), (9001, 2, 7, 385, 640, [1, 4, 6])]


def _inputs(g, n, experts, i, o, dtype):
    return (randn(g, n, i, dtype=dtype), (randn(g, experts, o, i) / i ** 0.5).to(dtype),
            randn(g, experts, o, dtype=dtype), randn(g, n, o, dtype=dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("tokens,topk,experts,i,o,to", SHAPES)
def test_forward_and_gradients(tokens, topk, experts, i, o, to, dtype):
    for drop in (0.0, 0.25):
        g = gen(tokens * i + o)
        _, offsets, _, _ = routed(tokens + i, tokens, topk, experts, drop, to)
        n, kept = tokens * topk, int(offsets[-1])
        xs, w, b, gys = _inputs(g, n, experts, i, o, dtype)
        xs[kept:] = float("nan")  # rows of no expert count for nothing
        gys[kept:] = float("nan")
        for bias in (b, None):
            ys = torch.full((n, o), 5.0, dtype=dtype, device=DEV)
            gs.gs_expert_linear_fwd(xs, offsets, w, bias, out=ys)
            ref, slack = linear_ref(xs, offsets, w, bias)
            check(ys, ref, slack, "ys")
            assert not bool(ys[kept:].any())
        got = gs.gs_expert_linear_bwd(gys, xs, offsets, w)
        refs, slacks = linear_bwd_ref(gys, xs, offsets, w)
        for t, r, s, name in zip(got, refs, slacks, ("grad_xs", "grad_weight", "grad_bias")):
            check(t, r, s, name)
        again = gs.gs_expert_linear_bwd(gys, xs, offsets, w, bias=False, input=False)
        assert again[0] is None and again[2] is None and torch.equal(again[1], got[1])


def test_no_rows():
    offsets = torch.zeros(4, dtype=torch.int32, device=DEV)
    w = torch.ones((3, 16, 32), device=DEV)
    xs = torch.empty((0, 32), device=DEV)
    assert gs.gs_expert_linear_fwd(xs, offsets, w).shape == (0, 16)
    gx, gw, gb = gs.gs_expert_linear_bwd(torch.empty((0, 16), device=DEV), xs, offsets, w)
    assert gx.shape == (0, 32) and not bool(gw.any()) and not bool(gb.any())


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows", [5, 600, 30000])
def test_rows_of_no_expert_only(rows, dtype):
    """Every pair dropped: zeros whatever the rows hold."""
    offsets = torch.zeros(4, dtype=torch.int32, device=DEV)
    nan = lambda *s: torch.full(s, float("nan"), dtype=dtype, device=DEV)
    w = randn(gen(1), 3, 264, 384, dtype=dtype)
    ys = gs.gs_expert_linear_fwd(nan(rows, 384), offsets, w, w[:, :, 0].contiguous())
    assert ys.shape == (rows, 264) and not bool(ys.any())
    for t in gs.gs_expert_linear_bwd(nan(rows, 264), nan(rows, 384), offsets, w):
        assert not bool(t.any())


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("tokens", [3, 2000])
def test_captured_in_a_graph(tokens, dtype):
    """The calls neither synchronise nor allocate on their own: a layer and
    its backward are captured once and replayed on new inputs."""
    g = gen(12)
    ids, offsets, _, _ = routed(12, tokens, 2, 4, 0.1)
    x, gy = randn(g, tokens, 72, dtype=dtype), randn(g, tokens, 40, dtype=dtype)
    w = (randn(g, 4, 40, 72) / 72 ** 0.5).to(dtype)
    p = torch.softmax(randn(g, tokens, 2), 1)

    def layer():
        n, mean, rstd = gs.gs_layer_norm_fwd(x)
        off, _, slots = gs.gs_expert_sort(ids, 4)
        xs = gs.gs_expert_dispatch(n, slots, off)
        ys = gs.gs_expert_linear_fwd(xs, off, w)
        y = gs.gs_expert_combine(ys, slots, p)
        gys, gp = gs.gs_expert_combine_bwd(gy, ys, slots, p, off)
        gxs, gw, gb = gs.gs_expert_linear_bwd(gys, xs, off, w)
        gx, _, _ = gs.gs_layer_norm_bwd(gs.gs_expert_combine(gxs, slots), x, None, mean, rstd)
        return y, gp, gw, gb, gx

    layer()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer()
    for seed in (1, 2):
        x.copy_(randn(gen(seed), tokens, 72, dtype=dtype))
        ids.copy_(routed(seed, tokens, 2, 4, 0.2)[0])
        graph.replay()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, layer()))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("tokens", [6, 400])
def test_infinity_and_nan_stay_in_their_rows_and_experts(tokens, dtype):
    g = gen(2)
    _, offsets, _, _ = routed(2, tokens, 2, 3, 0.0)
    xs, w, b, gys = _inputs(g, 2 * tokens, 3, 64, 128, dtype)
    clean = gs.gs_expert_linear_fwd(xs, offsets, w, b)
    bad = int(offsets[1]) + 1  # the second expert's second row
    xs[bad, 3] = float("nan")
    ys = gs.gs_expert_linear_fwd(xs, offsets, w, b)
    keep = torch.arange(2 * tokens, device=DEV) != bad
    assert torch.equal(ys[keep], clean[keep]) and bool(torch.isnan(ys[bad]).all())
    gw = gs.gs_expert_linear_bwd(gys, xs, offsets, w)[1]
    assert bool(torch.isfinite(gw[0]).all()) and bool(torch.isfinite(gw[2]).all())
    assert bool(torch.isnan(gw[1, :, 3]).all()) and int(torch.isnan(gw).sum()) == 128


@pytest.mark.parametrize("shift", [1, 3])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_bases_off_any_vector_boundary(shift, dtype):
    """Arrays that begin `shift` elements into an allocation."""
    g = gen(3)
    _, offsets, _, _ = routed(3, 150, 2, 3, 0.1)

    def moved(t):
        flat = torch.empty(t.numel() + shift, dtype=t.dtype, device=DEV)[shift:]
        flat.copy_(t.reshape(-1))
        return flat.reshape(t.shape)

    xs, w, b, gys = (moved(t) for t in _inputs(g, 300, 3, 128, 64, dtype))
    out = moved(torch.zeros((300, 64), dtype=dtype, device=DEV))
    ref, slack = linear_ref(xs, offsets, w, b)
    check(gs.gs_expert_linear_fwd(xs, offsets, w, b, out=out), ref, slack, "ys")
    refs, slacks = linear_bwd_ref(gys, xs, offsets, w)
    for t, r, s in zip(gs.gs_expert_linear_bwd(gys, xs, offsets, w), refs, slacks):
        check(t, r, s, "gradients")


def test_wide_range_in_32_bits():
    """float32 operands keep their 24 bits: values over 60 binades, within
    the bound of a float32 sum."""
    g = gen(4)
    _, offsets, _, _ = routed(4, 300, 1, 2, 0.0)
    xs, w, b, gys = _inputs(g, 300, 2, 96, 64, torch.float32)
    xs *= torch.exp2(torch.randint(-30, 30, xs.shape, generator=g, device=DEV).float())
    ref, slack = linear_ref(xs, offsets, w, None)
    check(gs.gs_expert_linear_fwd(xs, offsets, w), ref, slack, "ys")


@pytest.mark.parametrize("tokens,experts,i,o", [(3000, 2, 2056, 264), (12000, 2, 40, 520),
                                                (60, 4, 1500, 300)])
def test_float32_sums_stay_float32(tokens, experts, i, o):
    """Over thousands of terms of random sign a float32 sum is off by about
    2^-25 sqrt(terms / 2) of its size (each partial sum rounds); 1e-6 of the
    whole array's norm is what any order of 2000 terms keeps, and what sums
    that only ever cut off do not (3.8e-6 over 5000 terms)."""
    g = gen(9)
    _, offsets, _, _ = routed(9, tokens, 1, experts, 0.0)
    xs, w, b, gys = _inputs(g, tokens, experts, i, o, torch.float32)
    ref, _ = linear_ref(xs, offsets, w, b)
    refs, _ = linear_bwd_ref(gys, xs, offsets, w)
    got = (gs.gs_expert_linear_fwd(xs, offsets, w, b),
           *gs.gs_expert_linear_bwd(gys, xs, offsets, w))
    for t, r in zip(got, (ref, *refs)):
        assert float((t.double() - r).norm()) <= 1e-6 * float(r.norm())


def test_gradient_against_differences():
    """Linear in each argument: a difference of any width is the gradient up
    to the forward's rounding (1e-6 of its terms)."""
    g = gen(5)
    _, offsets, _, _ = routed(5, 90, 2, 4, 0.1)
    xs, w, b, gys = _inputs(g, 180, 4, 40, 56, torch.float32)
    grads = gs.gs_expert_linear_bwd(gys, xs, offsets, w)
    loss = lambda *a: float((gs.gs_expert_linear_fwd(a[0], offsets, a[1], a[2]).double()
                             * gys.double()).sum())
    for k, grad in enumerate(grads):
        args = [xs, w, b]
        v = randn(g, *args[k].shape)
        args[k] = args[k] + v
        up = loss(*args)
        args[k] = args[k] - 2 * v
        diff = (up - loss(*args)) / 2
        want = float((grad.double() * v.double()).sum())
        assert abs(diff - want) <= 1e-5 * float(grad.norm() * v.norm())


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_repeatability_and_another_stream(dtype):
    g = gen(6)
    _, offsets, _, _ = routed(6, 3000, 2, 3, 0.1)
    xs, w, b, gys = _inputs(g, 6000, 3, 256, 320, dtype)

    def passes(stream):
        return (gs.gs_expert_linear_fwd(xs, offsets, w, b, stream=stream),
                *gs.gs_expert_linear_bwd(gys, xs, offsets, w, stream=stream))

    first = passes(None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = passes(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, c) for a, c in zip(first, second))


def test_offsets_beyond_32_bits():
    n, i, o = 2 ** 21 + 77, 1032, 16
    offsets = torch.tensor([0, n - 200, n - 3], dtype=torch.int32, device=DEV)
    xs = torch.zeros((n, i), dtype=torch.bfloat16, device=DEV)  # 2.16e9 elements
    g = gen(8)
    xs[-400:] = randn(g, 400, i, dtype=torch.bfloat16)
    w = randn(g, 2, o, i, dtype=torch.bfloat16)
    ys = gs.gs_expert_linear_fwd(xs, offsets, w)
    tail = torch.tensor([0, 200, 397], dtype=torch.int32, device=DEV)
    ref, slack = linear_ref(xs[-400:], tail, w, None)
    check(ys[-400:], ref, slack, "ys")
    assert not bool(ys[:-400].any())
    gys = torch.zeros((n, o), dtype=torch.bfloat16, device=DEV)
    gys[-400:] = randn(g, 400, o, dtype=torch.bfloat16)
    got = gs.gs_expert_linear_bwd(gys, xs, offsets, w)
    refs, slacks = linear_bwd_ref(gys[-400:], xs[-400:], tail, w)
    check(got[0][-400:], refs[0], slacks[0], "grad_xs")
    check(got[1], refs[1], slacks[1], "grad_weight")
    check(got[2], refs[2], slacks[2], "grad_bias")


def test_offsets_outside_the_rows_are_clamped_and_reported():
    build.build()
    _, offsets, _, _ = routed(8, 100, 2, 4, 0.0)
    xs, w, b, gys = _inputs(gen(8), 200, 4, 64, 64, torch.bfloat16)
    good = gs.gs_expert_linear_fwd(xs, offsets, w, b)
    for place, value in ((4, 10 ** 6), (2, -5), (3, 10 ** 6)):
        bad = offsets.clone()
        bad[place] = value
        for lib, code in ((gs.LIB_PATH, 0), (gs.LIB_DEBUG_PATH, 9)):
            with gs.library(lib):
                st = gs.new_status(DEV)
                ys = gs.gs_expert_linear_fwd(xs, offsets, w, b, d_status=st)
                gs.check_status(st)
                assert torch.equal(ys, good)
                for call in (
                        lambda st: gs.gs_expert_linear_fwd(xs, bad, w, b, d_status=st),
                        lambda st: gs.gs_expert_linear_bwd(gys, xs, bad, w, d_status=st)):
                    st = gs.new_status(DEV)
                    call(st)
                    assert int(st.item()) == code


def test_refusals():
    xs = torch.zeros((6, 8), device=DEV)
    offsets = torch.tensor([0, 3, 6], dtype=torch.int32, device=DEV)
    w = torch.zeros((2, 5, 8), device=DEV)
    for bad in (lambda: gs.gs_expert_linear_fwd(xs, offsets, w[:, :, :7].contiguous()),
                lambda: gs.gs_expert_linear_fwd(xs, offsets, w.half()),
                lambda: gs.gs_expert_linear_fwd(xs, offsets[:2], w),
                lambda: gs.gs_expert_linear_fwd(xs, offsets.long(), w),
                lambda: gs.gs_expert_linear_fwd(xs, offsets, w, torch.zeros(5, device=DEV)),
                lambda: gs.gs_expert_linear_fwd(xs, offsets, w.transpose(1, 2)),
                lambda: gs.gs_expert_linear_bwd(xs, xs, offsets, w),
                lambda: gs.gs_expert_linear_fwd(xs.double(), offsets, w)):
        with pytest.raises(ValueError):
            bad()
