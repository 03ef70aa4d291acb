"""Argument checks of the feature-head calls: found on the host, before any
CUDA call, so they answer without a GPU."""

import ctypes as ct

import pytest

P = ct.c_void_p
F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    from tile_gaussian_splat_gb300 import binding, build
    build.build()
    return binding.lib()


def test_layer_norm(lib):
    def fwd(x=8, ldx=16, w=8, b=8, rows=4, ch=16, dt=F32, pt=F32, eps=1e-5, y=8, ldy=16, m=8,
            r=8):
        return lib.gs_layer_norm_fwd(P(x), ldx, P(w), P(b), rows, ch, dt, pt, eps, P(y), ldy,
                                     P(m), P(r), None)

    for bad in (dict(x=0), dict(x=2), dict(ldx=15), dict(rows=-1), dict(ch=0), dict(ch=16385),
                dict(dt=3), dict(pt=F16), dict(dt=F16, pt=BF16), dict(eps=-1.0),
                dict(eps=float("nan")), dict(y=0), dict(ldy=8), dict(m=0), dict(r=0),
                dict(w=6), dict(b=5)):
        assert fwd(**bad) == 1, bad
    assert fwd(rows=0, x=0, y=0) == 0  # nothing to do

    def bwd(gy=8, ldgy=16, x=8, m=8, rows=4, gx=8, ldgx=16, gw=8, gb=8, ws=8, n=1 << 30):
        return lib.gs_layer_norm_bwd(P(gy), ldgy, P(x), 16, P(8), P(m), P(8), rows, 16, F32, F32,
                                     P(gx), ldgx, P(gw), P(gb), P(ws), n, None)

    for bad in (dict(gy=0), dict(ldgy=3), dict(x=0), dict(m=0), dict(rows=-2), dict(ldgx=3),
                dict(gw=3), dict(gb=1)):
        assert bwd(**bad) == 1, bad
    assert bwd(ws=0) == 4 and bwd(n=16) == 4
    assert bwd(gx=0, gw=0, gb=0, ws=0, n=0) == 0  # no output asked for
    assert lib.gs_layer_norm_bwd_workspace_size(-1, 16) == 0
    assert lib.gs_layer_norm_bwd_workspace_size(100, 16) >= 128


def test_expert_sort(lib):
    def sort(ids=8, tokens=4, topk=2, experts=8, off=8, order=8, slots=8, ws=8, n=1 << 30):
        return lib.gs_expert_sort(P(ids), tokens, topk, experts, P(off), P(order), P(slots),
                                  P(ws), n, None)

    for bad in (dict(ids=0), dict(tokens=-1), dict(topk=0), dict(topk=65), dict(experts=0),
                dict(experts=1025), dict(off=0), dict(order=0), dict(slots=0), dict(ids=6),
                dict(tokens=1 << 30)):
        assert sort(**bad) == 1, bad
    assert sort(tokens=100000, ws=0) == 4 and sort(tokens=100000, n=100) == 4
    assert lib.gs_expert_sort_workspace_size(4, 0, 8) == 0
    assert lib.gs_expert_sort_workspace_size(100000, 2, 8) > 0


def test_rows(lib):
    def dispatch(x=8, ldx=16, slots=8, off=8, tokens=4, topk=2, experts=8, ch=16, dt=F32, xs=8):
        return lib.gs_expert_dispatch(P(x), ldx, P(slots), P(off), tokens, topk, experts, ch, dt,
                                      P(xs), None, None)

    for bad in (dict(x=0), dict(ldx=15), dict(slots=0), dict(off=0), dict(tokens=-1),
                dict(ch=0), dict(ch=65537), dict(dt=-1), dict(xs=0), dict(xs=2),
                dict(experts=2000)):
        assert dispatch(**bad) == 1, bad
    assert dispatch(tokens=0, x=0, slots=0, xs=0) == 0

    def combine(ys=8, slots=8, w=8, tokens=4, topk=2, ch=16, dt=BF16, y=8, ldy=16):
        return lib.gs_expert_combine(P(ys), P(slots), P(w), tokens, topk, ch, dt, P(y), ldy,
                                     None, None)

    for bad in (dict(ys=0), dict(slots=0), dict(w=2), dict(y=0), dict(ldy=15), dict(topk=0),
                dict(dt=9), dict(ys=9)):
        assert combine(**bad) == 1, bad

    def bwd(gy=8, ldgy=16, ys=8, slots=8, w=8, off=8, gys=8, gw=8):
        return lib.gs_expert_combine_bwd(P(gy), ldgy, P(ys), P(slots), P(w), P(off), 4, 2, 8, 16,
                                         F16, P(gys), P(gw), None, None)

    for bad in (dict(gy=0), dict(ldgy=2), dict(ys=0), dict(slots=0), dict(off=0), dict(gys=0),
                dict(gw=6), dict(w=1)):
        assert bwd(**bad) == 1, bad


def test_expert_linear(lib):
    def fwd(xs=16, off=8, w=16, b=16, rows=4, experts=2, i=8, o=8, dt=BF16, ys=16):
        return lib.gs_expert_linear_fwd(P(xs), P(off), P(w), P(b), rows, experts, i, o, dt, P(ys),
                                        None, 0, None, None)

    for bad in (dict(xs=0), dict(off=0), dict(off=6), dict(w=0), dict(b=1), dict(rows=-1),
                dict(rows=1 << 31), dict(experts=0), dict(experts=1025), dict(i=0), dict(o=0),
                dict(i=65537), dict(dt=4), dict(ys=0)):
        assert fwd(**bad) == 1, bad
    assert fwd(rows=0, xs=0, w=0, ys=0) == 0

    def bwd(gys=16, xs=16, off=8, w=16, rows=4, gx=16, gw=16, gb=16, ws=16, n=1 << 30):
        return lib.gs_expert_linear_bwd(P(gys), P(xs), P(off), P(w), rows, 2, 8, 8, BF16, P(gx),
                                        P(gw), P(gb), P(ws), n, None, None)

    for bad in (dict(gys=0), dict(xs=0), dict(off=0), dict(w=0), dict(gx=1), dict(gw=1), dict(gw=0),
                dict(gb=1), dict(rows=-1)):
        assert bwd(**bad) == 1, bad
    assert bwd(ws=0) == 4 and bwd(ws=8) == 4 and bwd(n=16) == 4  # missing, misaligned, small
    # float32 and rows of odd length are laid out in the workspace, unless there are few rows
    size = lib.gs_expert_linear_fwd_workspace_size
    assert size(1000, 2, 64, 32, BF16, 1) == 0 and size(1000, 2, 64, 32, BF16, 0) > 0
    assert size(1000, 2, 63, 32, F16, 1) > 0 and size(1000, 2, 64, 32, F32, 1) > 0
    assert size(1000, 0, 64, 32, F32, 1) == 0 and size(2, 2, 63, 32, F32, 0) == 0
    assert fwd(rows=1000, dt=F32) == 4 and fwd(rows=1000, i=7) == 4 and fwd(rows=1000, xs=18) == 4
    assert fwd(dt=F32, rows=(1 << 31) // 3 + 1) == 1
