"""float32 products of few terms: as exact as sums of float32 products, one
term included."""

import pytest
import torch

from head_util import DEV, gen, linear_bwd_ref
from tile_gaussian_splat_gb300 import binding as gs

pytestmark = pytest.mark.gpu

# In float32 a product rounds by 2^-24 of it (here: the plane pairs left out are
# below that) and n terms leave n partial sums, each off by 2^-23 at most.
UNIT = 2.0 ** -23
# whose upper eight bits are followed by ones (cut off) or just above half
WORST = (1 + 2.0 ** -7 - 2.0 ** -23, 1 + 2.0 ** -8 + 2.0 ** -17, 2 - 2.0 ** -23, 1 + 2.0 ** -8)


def _values(g, kind, *shape):
    u = torch.rand(shape, generator=g, device=DEV) + 1
    if kind == "worst":
        pick = torch.randint(len(WORST), shape, generator=g, device=DEV)
        return torch.tensor(WORST, device=DEV)[pick]
    if kind == "signed":
        return u * (torch.randint(2, shape, generator=g, device=DEV) * 2 - 1)
    return u


def _check(got, ref, size, n):
    over = (got.double() - ref).abs() - (n + 1) * UNIT * size
    assert float(over.max()) <= 0, f"{float((over / size).max()) / UNIT:.3g} units over"


@pytest.mark.parametrize("kind", ["worst", "positive", "signed"])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 16, 17])
def test_over_features(n, kind):
    g = gen(n)
    offsets = torch.tensor([0, 1500], dtype=torch.int32, device=DEV)
    x, w = _values(g, kind, 1500, n), _values(g, kind, 1, 200, n)
    _check(gs.gs_expert_linear_fwd(x, offsets, w), x.double() @ w[0].double().t(),
           x.double().abs() @ w[0].double().abs().t(), n)
    wt = w.transpose(1, 2).contiguous()
    gx = gs.gs_expert_linear_bwd(x, x.new_zeros(1500, 200), offsets, wt)[0]
    _check(gx, x.double() @ wt[0].double(), x.double().abs() @ wt[0].double().abs(), n)


@pytest.mark.parametrize("kind", ["worst", "positive", "signed"])
def test_over_rows(kind):
    g = gen(4)
    counts = torch.arange(200, device=DEV) % 5
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    rows = int(offsets[-1])
    x, gy = _values(g, kind, rows, 72), _values(g, kind, rows, 40)
    w = torch.zeros((200, 40, 72), device=DEV)
    gw, gb = gs.gs_expert_linear_bwd(gy, x, offsets, w, input=False)[1:]
    (_, rw, rb), _ = linear_bwd_ref(gy, x, offsets, w)
    (_, sw, sb), _ = linear_bwd_ref(gy.abs(), x.abs(), offsets, w)
    n = counts.double()
    _check(gw, rw, sw + (sw == 0), n[:, None, None])
    _check(gb, rb, sb + (sb == 0), n[:, None])
