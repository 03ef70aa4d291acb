"""The example that trains splat features through the expert head: its
gradients equal those of the same network written in torch in 64 bits, and
its loss falls."""

import importlib.util
import os

import pytest
import torch

from conftest import ROOT
from head_util import gen, randn

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(ROOT, "examples", "feature_head.py")
    spec = importlib.util.spec_from_file_location("feature_head", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _plain(head, x, reached):
    """The head in 64 bits, with autograd; the same choice of experts."""
    p = {k: v.double().requires_grad_() for k, v in head.params.items()}
    x = x.double().requires_grad_()
    mean = x.mean(-1, keepdim=True)
    var = ((x - mean) ** 2).mean(-1, keepdim=True)
    n = (x - mean) / torch.sqrt(var + 1e-5) * p["norm_w"] + p["norm_b"]
    rows = n.reshape(-1, n.shape[-1])
    logits = rows @ p["router"].t()
    ids = head.kept[4]
    weights = torch.softmax(logits.gather(1, ids), 1)
    y = 0
    for j in range(ids.shape[1]):
        h = torch.relu(torch.einsum("rhf,rf->rh", p["w1"][ids[:, j]], rows) + p["b1"][ids[:, j]])
        o = torch.einsum("roh,rh->ro", p["w2"][ids[:, j]], h) + p["b2"][ids[:, j]]
        y = y + weights[:, j:j + 1] * o
    y = y * reached.reshape(-1, 1)
    return x, p, y.reshape(*x.shape[:-1], -1)


def test_gradients_of_the_whole_head():
    ex = _example()
    head = ex.FeatureHead(24, 40, 6, 5, seed=3)
    g = gen(3)
    image = randn(g, 2, 20, 30, 27)
    reached = torch.rand((2, 20, 30), generator=g, device=image.device) > 0.2
    x = image[..., 3:]
    y = head.forward(x, reached)
    xr, p, out = _plain(head, x, reached)
    ref = out.detach()
    # 24- and 40-term sums of float32: a relative 1e-5 is over 20 times their rounding
    assert float((y.double() - ref).norm()) <= 1e-5 * float(ref.norm())
    gy = randn(g, *y.shape)
    grad_image = torch.full_like(image, 9.0)
    head.backward(gy * reached[..., None], grad_image[..., 3:])
    out.backward(gy.double() * reached[..., None])
    assert bool((grad_image[..., :3] == 9).all())
    for got, want in ((grad_image[..., 3:], xr.grad),
                      *((head.grads[k], p[k].grad) for k in head.grads)):
        assert float((got.double() - want).norm()) <= 1e-4 * float(want.norm())


def test_training_reduces_the_loss():
    losses = _example().train(steps=25)
    assert all(l == l for l in losses) and losses[-1] < 0.6 * losses[0]
