"""Host side of the feature-head calls on stand-ins for the CUDA runtime
(fake_runtime.cpp): workspace sizes and launches, without a GPU and the same
with one."""

import ctypes as ct
import itertools
import os
import re
import subprocess

import pytest

from conftest import ROOT
from tile_gaussian_splat_gb300 import binding, build

F32, F16, BF16 = 0, 1, 2
P = ct.c_void_p


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    build.build()
    objs = [os.path.join(build.BUILD, "release", os.path.basename(s) + ".o")
            for s in build.sources()]
    if not all(os.path.exists(o) for o in objs):
        build.build(force=True, debug=False)
    fake = os.path.join(ROOT, "tests", "fake_runtime.cpp")
    with open(fake) as f:
        wraps = sorted(set(re.findall(r"__wrap_(\w+)", f.read())))
    out = str(tmp_path_factory.mktemp("fake") / "libgs_host.so")
    subprocess.run([build._nvcc(), "-shared", "-cudart", "static", "-Xcompiler", "-fPIC", fake,
                    *objs, "-o", out, *(f"-Xlinker=--wrap={w}" for w in wraps)], check=True,
                   capture_output=True)
    L = ct.CDLL(out)
    for name, (res, args) in binding.SIGNATURES.items():
        fn = getattr(L, name)
        fn.restype, fn.argtypes = res, args
    L.fake_launches.restype = L.fake_blocks.restype = ct.c_int64
    L.fake_use(0, 0)
    return L


ALIGNED, SHIFTED = 1 << 20, (1 << 20) + 4  # elements of every type begin at both


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("i,o", [(128, 64), (64, 32), (8, 8), (63, 64), (64, 63), (131, 259)])
def test_the_queried_workspace_is_enough_whichever_array_is_misaligned(lib, i, o, dtype):
    """`aligned` = 0 says that some array is off a 16-byte boundary, not which;
    the size it gets serves every case, and that of `aligned` = 1 the aligned
    one."""
    for rows, experts in itertools.product(
            (1, 2, 16, 17, 20, 100, 128, 512, 1000, 1024, 1025, 5000), (1, 2, 8, 64, 1024)):
        for places in itertools.product((ALIGNED, SHIFTED), repeat=3):
            whole = all(p == ALIGNED for p in places)
            gys, xs, w = places
            n = lib.gs_expert_linear_fwd_workspace_size(rows, experts, i, o, dtype,
                                                        int(xs == w == ALIGNED))
            rc = lib.gs_expert_linear_fwd(P(xs), P(ALIGNED), P(w), None, rows, experts, i, o,
                                          dtype, P(ALIGNED), P(ALIGNED), n, None, None)
            assert rc == 0, ("forward", rows, experts, places)
            n = lib.gs_expert_linear_bwd_workspace_size(rows, experts, i, o, dtype, int(whole))
            rc = lib.gs_expert_linear_bwd(P(gys), P(xs), P(ALIGNED), P(w), rows, experts, i, o,
                                          dtype, P(ALIGNED), P(ALIGNED), P(ALIGNED), P(ALIGNED),
                                          n, None, None)
            assert rc == 0, ("backward", rows, experts, places)


@pytest.mark.parametrize("dtype,planes", [(BF16, 1), (F16, 1), (F32, 3)])
def test_rows_up_to_where_the_kernels_row_numbers_fit(lib, dtype, planes):
    """Row numbers, and those of the planes of float32, are 32-bit and formed
    before they are cut to the last row of a tile, up to 256 rows behind it."""
    most = ((1 << 31) - 256) // planes
    for rows, code in ((most, 0), (most + 1, 1), ((1 << 31) // planes, 1)):
        n = lib.gs_expert_linear_fwd_workspace_size(rows, 1, 8, 8, dtype, 1)
        assert lib.gs_expert_linear_fwd(P(ALIGNED), P(ALIGNED), P(ALIGNED), None, rows, 1, 8, 8,
                                        dtype, P(ALIGNED), P(ALIGNED), n, None, None) == code
        n = lib.gs_expert_linear_bwd_workspace_size(rows, 1, 8, 8, dtype, 1)
        assert lib.gs_expert_linear_bwd(P(ALIGNED), P(ALIGNED), P(ALIGNED), P(ALIGNED), rows, 1, 8,
                                        8, dtype, P(ALIGNED), P(ALIGNED), P(ALIGNED), P(ALIGNED),
                                        n, None, None) == code
        if code:
            assert n == 0


def _product(lib, rows=4096):
    n = lib.gs_expert_linear_bwd_workspace_size(rows, 4, 512, 512, BF16, 1)
    a = P(ALIGNED)
    return (lib.gs_expert_linear_fwd(a, a, a, None, rows, 4, 512, 512, BF16, a, None, 0, None,
                                     None),
            lib.gs_expert_linear_bwd(a, a, a, a, rows, 4, 512, 512, BF16, a, a, a, a, n, None,
                                     None))


def _sort(lib):
    a = P(ALIGNED)
    return lib.gs_expert_sort(a, 100, 2, 1024, a, a, a, None, 0, None)


ROWS = 1 << 20  # more than any device's resident blocks


def _norm(lib, ch=64):
    a = P(ALIGNED)
    return lib.gs_layer_norm_fwd(a, ch, None, None, ROWS, ch, F32, F32, 1e-5, a, ch, None, None,
                                 None)


def _dispatch(lib):
    a = P(ALIGNED)
    return lib.gs_expert_dispatch(a, 64, a, a, ROWS, 1, 8, 64, F32, a, None, None)


def _combine(lib):
    a = P(ALIGNED)
    return lib.gs_expert_combine(a, a, None, ROWS, 1, 64, F32, a, 64, None, None)


def test_kernels_are_set_up_on_every_device(lib):
    """A process may use several devices: what is set or found out about one
    is not taken for another's."""
    for device in (0, 1, 0, 3):
        lib.fake_use(device, 0)
        for _ in range(2):
            assert _product(lib) == (0, 0) and _sort(lib) == 0
        for call in (_norm, _dispatch, _combine):
            assert call(lib) == 0 and lib.fake_blocks() == 2 * (152 - 10 * device)
    # once a device
    calls, queries = lib.fake_attribute_calls(), lib.fake_queries()
    assert _product(lib) == (0, 0) and _sort(lib) == 0 and _norm(lib) == 0
    assert (lib.fake_attribute_calls(), lib.fake_queries()) == (calls, queries)
    lib.fake_use(0, 0)


def test_a_failed_query_is_asked_again(lib):
    lib.fake_use(4, 1)  # a device no call has used
    for call in (_norm, _dispatch, _combine):
        assert call(lib) == 0 and lib.fake_blocks() > 0  # some number of blocks does
    assert _product(lib) == (6, 6) and _sort(lib) == 6  # the limit is needed
    lib.fake_use(4, 0)
    assert _product(lib) == (0, 0) and _sort(lib) == 0
    for call in (_norm, _dispatch, _combine):
        assert call(lib) == 0 and lib.fake_blocks() == 2 * (152 - 40)
    lib.fake_use(0, 0)
