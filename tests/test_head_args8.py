"""Argument checks of the router's and the 8-bit rows' calls: found on the
host, before any CUDA call, so they answer without a GPU."""

import ctypes as ct

import pytest

P = ct.c_void_p
F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    from tile_gaussian_splat_gb300 import binding, build
    build.build()
    return binding.lib()


def test_route(lib):
    size = lib.gs_expert_route_workspace_size

    def fwd(x=8, ldl=8, keep=0, tokens=4, topk=2, experts=8, dt=F32, ids=8, w=8, c=8, l=8, ws=16,
            n=1 << 30):
        return lib.gs_expert_route_fwd(P(x), ldl, P(keep), tokens, topk, experts, dt, 1, P(ids),
                                       P(w), P(c), P(l), P(ws), n, None)

    for bad in (dict(x=0), dict(x=2), dict(ldl=7), dict(tokens=-1), dict(topk=0), dict(topk=9),
                dict(topk=65, experts=100, ldl=100), dict(experts=0), dict(experts=1025, ldl=1025),
                dict(dt=3), dict(dt=-1), dict(ids=0), dict(ids=6), dict(w=0), dict(w=1), dict(c=2),
                dict(l=3), dict(c=0), dict(tokens=1 << 30, topk=2)):
        assert fwd(**bad) == 1, bad
    assert size(8, 8) == 0  # a handful of tokens needs none
    assert fwd(tokens=9, ws=0) == 4 and fwd(tokens=9, ws=8) == 4 and fwd(tokens=9, n=16) == 4
    assert size(-1, 8) == 0 and size(10, 0) == 0 and size(10, 1025) == 0
    assert fwd(tokens=9, n=size(9, 8) - 1) == 4
    assert 0 < size(9, 1) <= size(1000, 8) <= size(10 ** 9, 1024) < 1 << 24

    def bwd(x=8, ldl=8, ids=8, c=8, gw=8, gl=8, tokens=4, topk=2, experts=8, dt=F16, g=8, ldg=8):
        return lib.gs_expert_route_bwd(P(x), ldl, P(ids), P(c), P(gw), P(gl), tokens, topk,
                                       experts, dt, 0, P(g), ldg, None, None)

    for bad in (dict(x=0), dict(x=3), dict(ldl=7), dict(ids=0), dict(c=0), dict(gw=2), dict(gl=1),
                dict(tokens=-1), dict(topk=0), dict(topk=9), dict(experts=0), dict(dt=7),
                dict(g=0), dict(g=1), dict(ldg=7)):
        assert bwd(**bad) == 1, bad
    assert bwd(tokens=0, x=0, ids=0, g=0) == 0  # nothing to do


def test_rows8(lib):
    def pack(x=16, ldx=40, rows=4, ch=40, dt=BF16, q=16, s=16):
        return lib.gs_rows_pack8(P(x), ldx, rows, ch, dt, P(q), P(s), None)

    def unpack(q=16, s=16, rows=4, ch=40, dt=BF16, y=16, ldy=40):
        return lib.gs_rows_unpack8(P(q), P(s), rows, ch, dt, P(y), ldy, None)

    for bad in (dict(x=0), dict(x=1), dict(ldx=39), dict(rows=-1), dict(ch=0), dict(ch=65537),
                dict(dt=3), dict(q=0), dict(q=8), dict(s=0), dict(s=2)):
        assert pack(**bad) == 1, bad
    for bad in (dict(q=0), dict(q=8), dict(s=0), dict(s=1), dict(rows=-1), dict(ch=0),
                dict(ch=65537), dict(dt=9), dict(y=0), dict(y=1), dict(ldy=39)):
        assert unpack(**bad) == 1, bad
    assert pack(rows=0, x=0, q=0, s=0) == 0 and unpack(rows=0, q=0, s=0, y=0) == 0


def test_linear8(lib):
    def fwd(x=16, xs=16, off=8, w=16, ws=16, b=16, rows=4, experts=2, i=40, o=24, dt=BF16, ys=16):
        return lib.gs_expert_linear8_fwd(P(x), P(xs), P(off), P(w), P(ws), P(b), rows, experts, i,
                                         o, dt, P(ys), None, None)

    for bad in (dict(x=0), dict(x=8), dict(xs=0), dict(xs=2), dict(off=0), dict(off=6), dict(w=0),
                dict(w=24), dict(ws=0), dict(b=1), dict(rows=-1), dict(rows=1 << 31),
                dict(experts=0), dict(experts=1025), dict(i=0), dict(i=65537), dict(o=0),
                dict(o=65537), dict(dt=4), dict(ys=0), dict(ys=1)):
        assert fwd(**bad) == 1, bad
    assert fwd(rows=0, x=0, w=0, ys=0) == 0

    def bwd(gys=16, x=16, xs=16, off=8, w=16, ws=16, rows=4, gx=16, gw=16, gb=16, room=16,
            n=1 << 30, dt=BF16):
        return lib.gs_expert_linear8_bwd(P(gys), P(x), P(xs), P(off), P(w), P(ws), rows, 2, 40, 24,
                                         dt, P(gx), P(gw), P(gb), P(room), n, None, None)

    for bad in (dict(gys=0), dict(gys=1), dict(x=0), dict(x=8), dict(xs=0), dict(off=0), dict(w=0),
                dict(w=8), dict(ws=3), dict(gx=1), dict(gw=1), dict(gw=0), dict(gb=1),
                dict(rows=-1), dict(dt=5)):
        assert bwd(**bad) == 1, bad
    size = lib.gs_expert_linear8_bwd_workspace_size
    for aligned in (0, 1):
        for dt in (F32, F16, BF16):
            n = size(5000, 2, 40, 24, dt, aligned)
            assert n > 0
            assert bwd(rows=5000, n=n - 1, dt=dt, gys=16 if aligned else 4) == 4
    assert bwd(room=0) == 4 and bwd(room=8) == 4
    assert size(5000, 2, 40, 0, BF16, 1) == 0
