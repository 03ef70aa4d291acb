"""Infinities and NaN in the experts' products: where the 64-bit form has an
infinity, a NaN or a number, so have the kernels, however many rows there are."""

import pytest
import torch

from head_util import DEV, TYPES, gen, randn
from tile_gaussian_splat_gb300 import binding as gs

pytestmark = pytest.mark.gpu

INF = float("inf")


def _same(got, ref, what):
    """The same infinities and NaN; the numbers beside them within the
    rounding of bfloat16 and of short sums."""
    assert bool((torch.isnan(got) == torch.isnan(ref)).all()), f"{what}: NaN"
    assert bool((torch.isinf(got) == torch.isinf(ref)).all()), f"{what}: infinities"
    assert bool((torch.sign(got.double()) == torch.sign(ref))[torch.isinf(ref)].all()), what
    ok = torch.isfinite(ref)
    err = (got.double() - ref).abs()[ok]
    assert float(err.max()) <= 0.01 * float(ref.abs()[ok].max()), what


def _spread(t, g, zeros):
    """Infinities of both signs in t's rows, also two of a row, and a NaN;
    values of eight bits (whose lower planes are 0) among the others."""
    rows, ch = t.shape
    t[::3] = t[::3].bfloat16().to(t.dtype)
    if zeros:
        t[:, 1] = 0
    t[2, 3] = INF
    t[rows // 2, 0] = -INF
    t[rows // 2 + 1, 1] = INF
    t[rows - 1, 2], t[rows - 1, ch - 1] = INF, -INF
    t[rows - 2, 4] = float("nan")
    return t


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows,i,o", [(12, 40, 24), (400, 64, 40), (3000, 264, 130), (900, 1100, 16)])
def test_products(rows, i, o, dtype):
    g = gen(rows)
    cut = rows // 3
    offsets = torch.tensor([0, cut, rows], dtype=torch.int32, device=DEV)
    xs, gys = randn(g, rows, i, dtype=dtype), randn(g, rows, o, dtype=dtype)
    w = (randn(g, 2, o, i) / i ** 0.5).to(dtype)
    b = randn(g, 2, o, dtype=dtype)
    for where in ("xs", "weight", "both", "grad_ys"):
        x, m, gy = xs.clone(), w.clone(), gys.clone()
        if where in ("xs", "both"):
            _spread(x, g, False)
            m[0, 5, 3] = 0  # an infinity against a zero is no number
        if where in ("weight", "both"):
            _spread(m[1], g, True)
        if where == "grad_ys":
            _spread(gy, g, True)
        ys = gs.gs_expert_linear_fwd(x, offsets, m, b)
        gx, gw, gb = gs.gs_expert_linear_bwd(gy, x, offsets, m)
        for e, r in enumerate((slice(0, cut), slice(cut, rows))):
            xd, md, gd = x[r].double(), m[e].double(), gy[r].double()
            _same(ys[r], xd @ md.t() + b[e].double(), f"{where}: ys")
            _same(gx[r], gd @ md, f"{where}: grad_xs")
            _same(gw[e], gd.t() @ xd, f"{where}: grad_weight")
            _same(gb[e], gd.sum(0), f"{where}: grad_bias")
