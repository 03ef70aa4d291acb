"""Host side of the router's and the 8-bit rows' calls on stand-ins for the
CUDA runtime (fake_runtime.cpp): workspace sizes, limits and launches, without
a GPU and the same with one."""

import itertools

import pytest

from test_head_host import ALIGNED, BF16, F16, F32, P, SHIFTED, lib  # noqa: F401


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("i,o", [(128, 64), (8, 8), (63, 64), (64, 63), (131, 259), (1024, 200)])
def test_the_queried_workspace_is_enough_however_the_gradient_lies(lib, i, o, dtype):  # noqa: F811
    a = P(ALIGNED)
    for rows, experts in itertools.product((1, 16, 17, 128, 1025, 5000, 100000), (1, 2, 64, 1024)):
        assert lib.gs_expert_linear8_fwd(a, a, a, a, a, None, rows, experts, i, o, dtype, a, None,
                                         None) == 0
        for gys in (ALIGNED, SHIFTED):
            n = lib.gs_expert_linear8_bwd_workspace_size(rows, experts, i, o, dtype,
                                                         int(gys == ALIGNED))
            for gx, gw, gb in ((a, a, a), (None, a, a), (a, None, None), (None, a, None)):
                rc = lib.gs_expert_linear8_bwd(P(gys), a, a, a, a, a, rows, experts, i, o, dtype,
                                               gx, gw, gb, a, n, None, None)
                assert rc == 0, (rows, experts, gys)


@pytest.mark.parametrize("dtype,planes", [(BF16, 1), (F16, 1), (F32, 3)])
def test_rows_up_to_where_the_kernels_row_numbers_fit(lib, dtype, planes):  # noqa: F811
    a = P(ALIGNED)
    most = ((1 << 31) - 256) // planes
    for rows, code in ((most, 0), (most + 1, 1), ((1 << 31) // planes, 1)):
        assert lib.gs_expert_linear8_fwd(a, a, a, a, a, None, rows, 1, 8, 8, dtype, a, None,
                                         None) == code
        n = lib.gs_expert_linear8_bwd_workspace_size(rows, 1, 8, 8, dtype, 1)
        assert lib.gs_expert_linear8_bwd(a, a, a, a, a, a, rows, 1, 8, 8, dtype, a, a, a, a, n,
                                         None, None) == code
        if code:
            assert n == 0


def _calls(lib):  # noqa: F811
    a = P(ALIGNED)
    rows = 1 << 20
    n = lib.gs_expert_route_workspace_size(rows, 16)
    yield lambda: lib.gs_expert_route_fwd(a, 16, None, rows, 2, 16, F32, 1, a, a, None, None,
                                          None, 0, None)
    yield lambda: lib.gs_expert_route_fwd(a, 16, None, rows, 2, 16, F32, 1, a, a, a, a, a, n, None)
    yield lambda: lib.gs_expert_route_bwd(a, 16, a, a, a, a, rows, 2, 16, F32, 1, a, 16, None, None)
    yield lambda: lib.gs_rows_pack8(a, 64, rows, 64, BF16, a, a, None)
    yield lambda: lib.gs_rows_unpack8(a, a, rows, 64, BF16, a, 64, None)


def _product(lib, rows, i=512, o=512):  # noqa: F811
    a = P(ALIGNED)
    return lib.gs_expert_linear8_fwd(a, a, a, a, a, a, rows, 4, i, o, BF16, a, None, None)


SHAPES = [(40000, 512, 512), (40000, 1024, 512), (100, 512, 512), (40000, 512, 64), (4, 512, 512)]


def test_kernels_are_set_up_on_every_device(lib):  # noqa: F811
    for device in (0, 2, 0, 5):
        lib.fake_use(device, 0)
        for shape in SHAPES:
            assert _product(lib, *shape) == 0
        for call in _calls(lib):
            assert call() == 0
    # once a device
    before = lib.fake_attribute_calls(), lib.fake_queries()
    for shape in SHAPES:
        assert _product(lib, *shape) == 0
    for call in _calls(lib):
        assert call() == 0
    assert (lib.fake_attribute_calls(), lib.fake_queries()) == before
    lib.fake_use(0, 0)


def test_a_failed_query_is_asked_again(lib):  # noqa: F811
    lib.fake_use(6, 1)  # a device no call has used
    for call in _calls(lib):
        assert call() == 0 and lib.fake_blocks() > 0  # some number of blocks does
    assert [_product(lib, *s) for s in SHAPES] == [6, 6, 6, 6, 0]  # the limit is needed
    lib.fake_use(6, 0)
    for call in _calls(lib):
        assert call() == 0
    assert [_product(lib, *s) for s in SHAPES] == [0] * 5
    lib.fake_use(0, 0)


def test_blocks_are_those_that_fit(lib):  # noqa: F811
    """Never more than a device holds at once, and no more than there is work."""
    lib.fake_use(0, 0)
    a = P(ALIGNED)
    assert lib.gs_rows_pack8(a, 64, 1 << 20, 64, BF16, a, a, None) == 0
    assert lib.fake_blocks() == 2 * 152
    assert lib.gs_rows_pack8(a, 64, 16, 64, BF16, a, a, None) == 0 and lib.fake_blocks() == 1
    assert _product(lib, 40000) == 0 and lib.fake_blocks() == 152
    assert lib.gs_expert_route_fwd(a, 16, None, 9, 2, 16, F32, 1, a, a, None, None, None, 0,
                                   None) == 0 and lib.fake_blocks() == 1
