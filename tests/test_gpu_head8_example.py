"""The example's head with 8-bit rows: it runs, and its gradients equal those of
the same network written in torch in 64 bits, with the rounding to 8 bits taken
over and passed over by the gradients."""

import pytest
import torch

from head8_util import values_ref
from head_util import gen, randn
from test_gpu_head_example import _example

pytestmark = pytest.mark.gpu


class _Through(torch.autograd.Function):
    """The rounded values; the gradient as if they were the others."""

    @staticmethod
    def forward(ctx, values, rounded):
        return rounded

    @staticmethod
    def backward(ctx, grad):
        return grad, None


def _plain(head, x):
    from tile_gaussian_splat_gb300 import binding as gs

    (_, _, _, rows8, _, ids, _, counts, _, slots, _, h8, w1, w2, _) = head.kept
    p = {k: v.double().requires_grad_() for k, v in head.params.items()}
    x = x.double().requires_grad_()
    mean = x.mean(-1, keepdim=True)
    var = ((x - mean) ** 2).mean(-1, keepdim=True)
    n = (x - mean) / torch.sqrt(var + 1e-5) * p["norm_w"] + p["norm_b"]
    rows = n.reshape(-1, n.shape[-1])
    D, H, E = rows.shape[1], p["w1"].shape[1], head.experts
    took = ids[:, 0] >= 0
    some = ids.clamp(min=0).long()
    probs = torch.softmax(rows @ p["router"].t(), 1) * took[:, None]
    chosen = probs.gather(1, some)
    weights = chosen / chosen.sum(1, keepdim=True).clamp(min=1e-300)
    pairs = counts[:E].double()
    balance = E * (pairs / pairs.sum() * probs.sum(0) / counts[E].double()).sum()
    through = _Through.apply
    xv = through(rows, values_ref(*gs.gs_rows_pack8(rows8), D))
    v1 = through(p["w1"], values_ref(*w1, D))
    v2 = through(p["w2"], values_ref(*w2, H))
    hv = values_ref(*h8, H)
    y = 0
    for j in range(ids.shape[1]):
        h = torch.einsum("rhf,rf->rh", v1[some[:, j]], xv) + p["b1"][some[:, j]]
        kept = hv[slots[:, j].clamp(min=0).long()]
        h = through(torch.where(kept > 0, h, 0.0), kept)
        o = torch.einsum("roh,rh->ro", v2[some[:, j]], h) + p["b2"][some[:, j]]
        y = y + weights[:, j:j + 1] * o * took[:, None]
    return x, p, y.reshape(*x.shape[:-1], -1), balance


def test_gradients_of_the_whole_head():
    ex = _example()
    head = ex.EightBitHead(24, 40, 6, 5, seed=3, balance=0.5)
    g = gen(3)
    image = randn(g, 2, 20, 30, 27)
    reached = torch.rand((2, 20, 30), generator=g, device=image.device) > 0.2
    x = image[..., 3:]
    y = head.forward(x, reached)
    xr, p, out, balance = _plain(head, x)
    ref = out.detach()
    # sums of at most 40 float32 terms: a relative 1e-5 is over 20 times their rounding
    assert float((y.double() - ref).norm()) <= 1e-5 * float(ref.norm())
    assert abs(float(head.balance_loss) - float(balance.detach())) <= 1e-5 * float(balance.detach())
    gy = randn(g, *y.shape) * reached[..., None]
    grad_image = torch.full_like(image, 9.0)
    head.backward(gy, grad_image[..., 3:])
    ((out * gy.double()).sum() + 0.5 * balance).backward()
    assert bool((grad_image[..., :3] == 9).all())
    for got, want in ((grad_image[..., 3:], xr.grad),
                      *((head.grads[k], p[k].grad) for k in head.grads)):
        assert float((got.double() - want).norm()) <= 1e-4 * float(want.norm())


def test_it_trains():
    ex = _example()
    losses = ex.train(steps=5, head_type=ex.EightBitHead)
    assert len(losses) == 5 and all(v == v for v in losses)


@pytest.mark.parametrize("call", ["gs_expert_linear8_fwd", "gs_expert_linear8_bwd",
                                  "gs_expert_route_bwd"])
def test_a_reported_error_stops_the_training(call, monkeypatch):
    from tile_gaussian_splat_gb300 import binding as gs

    ex = _example()
    made = []

    class Head(ex.EightBitHead):
        def __init__(self, *args, **kw):
            super().__init__(*args, **kw)
            made.append((self, {k: v.clone() for k, v in self.params.items()}))

    def reporting(*args, d_status=None, **kw):
        out = genuine(*args, d_status=d_status, **kw)
        if d_status is not None:
            d_status.fill_(5)  # as a wait that ran out does
        return out

    genuine = getattr(gs, call)
    monkeypatch.setattr(gs, call, reporting)
    with pytest.raises(gs.GsError, match="TIMEOUT"):
        ex.train(steps=1, head_type=Head)
    head, before = made[0]
    assert all(torch.equal(head.params[k], v) for k, v in before.items())
