"""Long sums of the experts' products stay float32 sums: terms of one sign,
where an accumulator that only ever cuts off falls behind in proportion to its
length, against the 64-bit sums."""

import pytest
import torch

from head_util import DEV, TYPES, gen
from tile_gaussian_splat_gb300 import binding as gs

pytestmark = pytest.mark.gpu

# A step of 16 terms cuts off a few units of the last place, 2^-23 of the sum
# so far (taken as four); sums of one sign are half their final size on
# average, and an accumulator takes at most 128 steps (float32: 32) before its
# sum is added, rounded to the nearest, to the running one.
BOUND = {torch.float32: 32 * 2 * 2.0 ** -23, torch.float16: 128 * 2 * 2.0 ** -23,
         torch.bfloat16: 128 * 2 * 2.0 ** -23}


def _positive(g, dtype, scale, *shape):
    return (torch.rand(shape, generator=g, device=DEV) * scale).to(dtype)


def _drift(got, ref):
    """Mean relative error beside the rounding of the output to its type."""
    return abs(float(((got.double() - ref.to(got.dtype).double()) / ref).mean()))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("depth", [4096, 32768, 65536])
def test_over_features(depth, dtype):
    g = gen(depth)
    rows, few = 600, 64
    offsets = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    x, w = _positive(g, dtype, 0.125, rows, depth), _positive(g, dtype, 0.004, 1, few, depth)
    y = gs.gs_expert_linear_fwd(x, offsets, w)
    assert _drift(y, x.double() @ w[0].double().t()) <= BOUND[dtype]
    # the input gradient sums over the outputs
    w = w.transpose(1, 2).contiguous()
    gx = gs.gs_expert_linear_bwd(x, _positive(g, dtype, 1.0, rows, few), offsets, w)[0]
    assert _drift(gx, x.double() @ w[0].double()) <= BOUND[dtype]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows,i,o", [(200000, 512, 1024), (60000, 2048, 2048), (150000, 96, 2000)])
def test_over_rows(rows, i, o, dtype):
    g = gen(rows + i)
    offsets = torch.tensor([0, rows // 3, rows], dtype=torch.int32, device=DEV)
    xs, gys = _positive(g, dtype, 1.0, rows, i), _positive(g, dtype, 8.0 / rows, rows, o)
    w = torch.zeros((2, o, i), dtype=dtype, device=DEV)
    _, gw, gb = gs.gs_expert_linear_bwd(gys, xs, offsets, w, input=False)
    for e, r in enumerate((slice(0, rows // 3), slice(rows // 3, rows))):
        assert _drift(gw[e], gys[r].double().t() @ xs[r].double()) <= BOUND[dtype]
        assert _drift(gb[e], gys[r].double().sum(0)) <= BOUND[dtype]
