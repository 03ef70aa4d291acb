"""Feature-head calls on arrays laid out, aligned or used in other ways than
fresh allocations on the current stream."""

import pytest
import torch

from head_util import DEV, TYPES, check, gen, linear_bwd_ref, linear_ref, randn, routed
from tile_gaussian_splat_gb300 import binding as gs

pytestmark = pytest.mark.gpu


def _shifted(t):
    """A contiguous copy that begins one element into an allocation."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:]
    flat.copy_(t.reshape(-1))
    return flat.reshape(t.shape)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows,experts", [(20, 2), (100, 8), (1000, 64), (3000, 3)])
def test_one_array_off_any_vector_boundary(rows, experts, dtype):
    """Each operand in turn, the others aligned: what one of them needs does
    not follow from another's alignment."""
    g = gen(rows)
    _, offsets, _, _ = routed(rows, rows, 1, experts, 0.1)
    arrays = [randn(g, rows, 128, dtype=dtype), (randn(g, experts, 64, 128) / 12).to(dtype),
              randn(g, rows, 64, dtype=dtype)]
    for k in range(3):
        xs, w, gys = (_shifted(t) if j == k else t for j, t in enumerate(arrays))
        ref, slack = linear_ref(xs, offsets, w, None)
        check(gs.gs_expert_linear_fwd(xs, offsets, w), ref, slack, "ys")
        refs, slacks = linear_bwd_ref(gys, xs, offsets, w)
        for t, r, s in zip(gs.gs_expert_linear_bwd(gys, xs, offsets, w), refs, slacks):
            check(t, r, s, "gradients")
