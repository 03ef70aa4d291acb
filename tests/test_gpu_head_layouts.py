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


def test_results_of_another_stream_share_no_memory_with_work_under_way():
    """The current stream still has writes to come into a block that it has
    freed; a call on another stream returns before them and keeps its result."""
    g = gen(21)
    x = randn(g, 1 << 14, 256)
    want = gs.gs_layer_norm_fwd(x, stats=False)[0].clone()
    side = torch.cuda.Stream()
    for _ in range(4):
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        block = torch.empty_like(x)
        y = z = torch.ones((4096, 4096), device=DEV)
        for _ in range(40):  # some milliseconds
            z = (z @ y) * 1e-4
        block.fill_(9.0)
        del block
        got = gs.gs_layer_norm_fwd(x, stats=False, stream=side)[0]
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        torch.cuda.current_stream().wait_stream(side)
        again = got + 0  # and the result is used on the current stream
        del got
        gs.gs_layer_norm_fwd(-x, stats=False, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(again, want)
