"""Layer norm of the feature head against its 64-bit form."""

import pytest
import torch

from head_util import DEV, TYPES, check, gen, norm_bwd_ref, norm_ref, randn, sliced
from tile_gaussian_splat_gb300 import binding as gs

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (1, 64), (5, 3), (7, 31), (129, 64), (64, 131), (33, 256), (40, 515),
          (1000, 1024), (9, 1023), (17, 2050), (6, 5000), (3, 16384), (4099, 24), (2500, 128),
          (70, 4096), (45, 2047), (31, 1500), (700, 4095), (20, 2048), (9, 3998)]


def _params(g, ch, p):
    return (1 + 0.1 * randn(g, ch)).to(p), randn(g, ch).to(p)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows,ch", SHAPES)
def test_forward_and_backward(rows, ch, dtype):
    for k, (pad, p) in enumerate([(0, dtype), (3, torch.float32), (8, dtype)]):
        g = gen(100 * rows + ch + k)
        x = sliced(randn(g, rows, ch, dtype=dtype) + randn(g, rows, 1, dtype=dtype), pad)
        w, b = _params(g, ch, p)
        y, mean, rstd = gs.gs_layer_norm_fwd(x, w, b, 1e-5)
        ry, rm, rr, sy, sm, sr = norm_ref(x, w, b, 1e-5)
        check(y, ry, sy, "y")
        check(mean, rm, sm, "mean")
        check(rstd, rr, sr, "rstd")
        gy = sliced(randn(g, rows, ch, dtype=dtype), pad)
        # the gradient goes into the channel slice of a wider image
        wide = torch.full((rows, ch + pad), 3.0, dtype=dtype, device=DEV)
        gx, gw, gb = gs.gs_layer_norm_bwd(gy, x, w, mean, rstd, out=wide[:, pad:])
        rx, rw, rb, sx, sw, sb = norm_bwd_ref(gy, x, w, mean, rstd)
        check(gx, rx, sx, "grad_x")
        check(gw, rw, sw, "grad_weight")
        check(gb, rb, sb, "grad_bias")
        assert gw.dtype == p and bool((wide[:, :pad] == 3).all())


def test_without_weight_bias_or_statistics():
    g = gen(1)
    x = randn(g, 77, 96)
    y, mean, rstd = gs.gs_layer_norm_fwd(x)
    ry, _, _, sy, _, _ = norm_ref(x, None, None, 1e-5)
    check(y, ry, sy, "y")
    y2, m2, r2 = gs.gs_layer_norm_fwd(x, stats=False)
    assert m2 is None and r2 is None and torch.equal(y, y2)
    gy = randn(g, 77, 96)
    gx, gw, gb = gs.gs_layer_norm_bwd(gy, x, None, mean, rstd)
    rx, rw, rb, sx, sw, sb = norm_bwd_ref(gy, x, None, mean, rstd)
    for got, ref, s in ((gx, rx, sx), (gw, rw, sw), (gb, rb, sb)):
        check(got, ref, s, "gradients")
    gx2, none1, none2 = gs.gs_layer_norm_bwd(gy, x, None, mean, rstd, params=False)
    assert torch.equal(gx, gx2) and none1 is None and none2 is None


def test_rows_without_spread_and_offsets_far_from_zero():
    x = torch.zeros((6, 64), device=DEV)
    x[1] = 3.0
    x[2] = 1e4
    x[3] = 1e4 + randn(gen(2), 64)
    x[4] = 1e18
    x[4, ::2] = -1e18
    y, mean, rstd = gs.gs_layer_norm_fwd(x, eps=1e-5)
    assert bool((y[:3] == 0).all())  # these means are exact
    assert float(rstd[0]) == pytest.approx(1e5 ** 0.5, rel=1e-6)
    ry, _, _, sy, _, _ = norm_ref(x, None, None, 1e-5)
    check(y[3:5], ry[3:5], sy[3:5], "y")
    # eps = 0 on a row without spread is 0 / 0, as the formula says
    assert bool(torch.isnan(gs.gs_layer_norm_fwd(x[:1], eps=0.0)[0]).all())


@pytest.mark.parametrize("ch", [64, 131, 1024, 4096])
def test_nan_and_infinity_stay_in_their_row(ch):
    g = gen(ch)
    x = randn(g, 40, ch)
    clean = gs.gs_layer_norm_fwd(x)[0]
    x[3, 5] = float("nan")
    x[17, 0] = float("inf")
    y = gs.gs_layer_norm_fwd(x)[0]
    keep = [r for r in range(40) if r not in (3, 17)]
    assert torch.equal(y[keep], clean[keep])
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(y[17]).all())


def test_no_rows():
    x = torch.empty((0, 33), device=DEV)
    w = torch.ones(33, device=DEV)
    y, mean, rstd = gs.gs_layer_norm_fwd(x, w, w)
    assert y.shape == (0, 33) and mean.shape == (0,)
    gx, gw, gb = gs.gs_layer_norm_bwd(x, x, w, mean, rstd)
    assert gx.shape == (0, 33) and bool((gw == 0).all()) and bool((gb == 0).all())


def test_image_shapes_and_repeatability():
    g = gen(9)
    image = randn(g, 2, 37, 53, 67)  # 3 colours and 64 features a pixel
    x = image[..., 3:]
    w, b = _params(g, 64, torch.float32)
    y, mean, rstd = gs.gs_layer_norm_fwd(x, w, b)
    assert y.shape == (2, 37, 53, 64) and mean.shape == (2, 37, 53)
    ry, _, _, sy, _, _ = norm_ref(x, w, b, 1e-5)
    check(y, ry, sy, "y")
    gy = randn(g, 2, 37, 53, 64)
    a = gs.gs_layer_norm_bwd(gy, x, w, mean, rstd)
    b2 = gs.gs_layer_norm_bwd(gy, x, w, mean, rstd)
    assert all(torch.equal(p, q) for p, q in zip(a, b2))


def test_offsets_beyond_32_bits():
    rows, ch = 2 ** 21 + 5, 1027
    x = torch.zeros((rows, ch), dtype=torch.float16, device=DEV)  # 2.15e9 elements
    x[-3:] = randn(gen(4), 3, ch, dtype=torch.float16)
    y, mean, rstd = gs.gs_layer_norm_fwd(x)
    ry, _, _, sy, _, _ = norm_ref(x[-3:], None, None, 1e-5)
    check(y[-3:], ry, sy, "y")
    assert not bool(y[:-3].any())
    gy = torch.zeros_like(x)
    gy[-3:] = randn(gen(5), 3, ch, dtype=torch.float16)
    gx, gw, gb = gs.gs_layer_norm_bwd(gy, x, None, mean, rstd)
    rx, rw, rb, sx, sw, sb = norm_bwd_ref(gy[-3:], x[-3:], None, mean[-3:], rstd[-3:])
    check(gx[-3:], rx, sx, "grad_x")
    check(gw, rw, sw, "grad_weight")
    check(gb, rb, sb, "grad_bias")
    assert not bool(gx[:-3].any())


def test_gradient_against_differences():
    """Central differences of the forward kernel along random directions:
    the forward's rounding (6e-8 a value, 1e3 values) over 2h = 0.02 and the
    cubic term h^2 together stay below 1e-3 of |gradient| |direction|."""
    g = gen(7)
    x = randn(g, 31, 48)
    w, b = _params(g, 48, torch.float32)
    gy = randn(g, 31, 48)
    _, mean, rstd = gs.gs_layer_norm_fwd(x, w, b)
    gx, gw, gb = gs.gs_layer_norm_bwd(gy, x, w, mean, rstd)
    loss = lambda x_, w_, b_: float((gs.gs_layer_norm_fwd(x_, w_, b_)[0].double()
                                     * gy.double()).sum())
    h = 0.01
    for k, (t, grad) in enumerate(((x, gx), (w, gw), (b, gb))):
        v = randn(g, *t.shape)
        args = [x, w, b]
        args[k] = t + h * v
        up = loss(*args)
        args[k] = t - h * v
        diff = (up - loss(*args)) / (2 * h)
        want = float((grad.double() * v.double()).sum())
        assert abs(diff - want) <= 1e-3 * float(grad.norm() * v.norm())


def test_on_another_stream():
    g = gen(11)
    x = randn(g, 4000, 256)
    gy = randn(g, 4000, 256)
    w, b = _params(g, 256, torch.float32)
    y, mean, rstd = gs.gs_layer_norm_fwd(x, w, b)
    grads = gs.gs_layer_norm_bwd(gy, x, w, mean, rstd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, m2, r2 = gs.gs_layer_norm_fwd(x, w, b, stream=side)
    grads2 = gs.gs_layer_norm_bwd(gy, x, w, m2, r2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, y2) and all(torch.equal(p, q) for p, q in zip(grads, grads2))


def test_refusals():
    x = torch.zeros((4, 8), device=DEV)
    w = torch.ones(8, device=DEV)
    stats = torch.zeros(4, device=DEV)
    for bad in (lambda: gs.gs_layer_norm_fwd(x.double()), lambda: gs.gs_layer_norm_fwd(x.t()),
                lambda: gs.gs_layer_norm_fwd(x, w[:7]), lambda: gs.gs_layer_norm_fwd(x, w.half()),
                lambda: gs.gs_layer_norm_fwd(x, w, w.half()),
                lambda: gs.gs_layer_norm_fwd(x.cpu()),
                lambda: gs.gs_layer_norm_fwd(x, out=torch.zeros((4, 9), device=DEV)),
                lambda: gs.gs_layer_norm_fwd(x[:1].expand(4, 8)),
                lambda: gs.gs_layer_norm_bwd(x.half(), x, w, stats, stats),
                lambda: gs.gs_layer_norm_bwd(x, x, w, stats[:3], stats)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(gs.GsError, match="INVALID_ARG"):
        gs.gs_layer_norm_fwd(x, eps=-1.0)
    with pytest.raises(gs.GsError, match="INVALID_ARG"):
        gs.gs_layer_norm_fwd(torch.zeros((1, 16385), device=DEV))
