"""Plain 64-bit forms of the feature-head operators and the error bounds the
GPU tests hold the kernels to.

Bounds.  An output is computed in float32 and rounded to its type once, so
its error is at most U[type] * |value| plus that of the float32 computation.
A sum of n products in float32, in any order, is off by at most
(n + 2) * 2^-23 * sum |products| (2^-23: each step may round or truncate).
"""

from __future__ import annotations

import numpy as np
import torch

DEV = "cuda:0"
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 1e-37, torch.float16: 2.0 ** -24, torch.bfloat16: 1e-37}
U32 = 2.0 ** -23
TYPES = [torch.float32, torch.float16, torch.bfloat16]


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def sliced(x, pad):
    """x as the last columns of a wider array whose other columns are 7."""
    wide = torch.full((*x.shape[:-1], x.shape[-1] + pad), 7.0, dtype=x.dtype, device=x.device)
    wide[..., pad:] = x
    return wide[..., pad:]


def check(got, ref, slack, what):
    """|got - ref| <= U |ref| + slack, elementwise (slack: the float32 part)."""
    assert got.shape == ref.shape, what
    err = (got.double() - ref).abs()
    allowed = U[got.dtype] * ref.abs() + slack * (1 + U[got.dtype]) + TINY[got.dtype]
    bad = ~(err <= allowed)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err - allowed).max()):.3g} "
        f"over at {float(err.max()):.3g}")


def norm_ref(x, weight, bias, eps):
    x = x.double()
    n = x.shape[-1]
    w = weight.double() if weight is not None else torch.ones((), dtype=torch.float64, device=DEV)
    b = bias.double() if bias is not None else torch.zeros((), dtype=torch.float64, device=DEV)
    mean = x.sum(-1, keepdim=True) / n
    d = x - mean
    rstd = 1 / torch.sqrt((d * d).sum(-1, keepdim=True) / n + eps)
    y = d * rstd * w + b
    # the mean is off by at most dm, which moves d by as much and the variance
    # by dm^2 (the sum of d is 0) beside its own rounding
    dm = (n + 2) * U32 * x.abs().sum(-1, keepdim=True) / n
    rel = 0.5 * ((n + 8) * U32 + (dm * rstd) ** 2) + 4 * U32
    slack = w.abs() * rstd * (dm + 2 * U32 * d.abs()) + (d * rstd * w).abs() * (rel + 4 * U32) \
        + 2 * U32 * b.abs()
    return y, mean[..., 0], rstd[..., 0], slack, dm[..., 0], (rel * rstd)[..., 0]


def norm_bwd_ref(gy, x, weight, mean, rstd):
    """For the given float32 statistics."""
    x, gy = x.double(), gy.double()
    n = x.shape[1]
    w = weight.double() if weight is not None else torch.ones((), dtype=torch.float64, device=DEV)
    r = rstd.double().reshape(-1, 1)
    mu = mean.double().reshape(-1, 1)
    xh = (x - mu) * r
    dxh = 4 * U32 * xh.abs()
    g = gy * w
    s0, s1 = g.sum(1, keepdim=True) / n, (g * xh).sum(1, keepdim=True) / n
    gx = r * (g - s0 - xh * s1)
    d0 = (n + 4) * U32 * g.abs().sum(1, keepdim=True) / n
    d1 = (n + 8) * U32 * (g * xh).abs().sum(1, keepdim=True) / n
    slack = r * (8 * U32 * (g.abs() + s0.abs() + (xh * s1).abs()) + d0 + xh.abs() * d1
                 + dxh * s1.abs())
    m = x.shape[0]
    gw, gb = (gy * xh).sum(0), gy.sum(0)
    sw = (m + 8) * U32 * (gy * xh).abs().sum(0)
    sb = (m + 8) * U32 * gy.abs().sum(0)
    return gx, gw, gb, slack, sw, sb


def sort_ref(ids, experts):
    flat = ids.cpu().numpy().reshape(-1)
    n = flat.size
    key = np.where((flat >= 0) & (flat < experts), flat, experts)
    order = np.argsort(key, kind="stable").astype(np.int32)
    offsets = np.searchsorted(key[order], np.arange(experts + 1)).astype(np.int32)
    slots = np.full(n, -1, np.int32)
    kept = int(offsets[-1])
    slots[order[:kept]] = np.arange(kept, dtype=np.int32)
    order[kept:] = -1
    return offsets, order, slots.reshape(ids.shape)


def routed(seed, tokens, topk, experts, drop=0.1, to=None):
    """(ids, offsets, order, slots) on the device; `to`: experts that get rows."""
    rng = np.random.default_rng(seed)
    pool = np.asarray(to if to is not None else np.arange(experts))
    ids = pool[rng.integers(0, pool.size, (tokens, topk))].astype(np.int32)
    ids[rng.random((tokens, topk)) < drop] = -1
    ids = torch.from_numpy(ids)
    plan = sort_ref(ids, experts)
    return (ids.to(DEV), *(torch.from_numpy(np.ascontiguousarray(p)).to(DEV) for p in plan))


def linear_ref(xs, offsets, weight, bias):
    off = offsets.tolist()
    E, o, i = weight.shape
    y = torch.zeros((xs.shape[0], o), dtype=torch.float64, device=DEV)
    slack = torch.zeros_like(y)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        a, w = xs[r].double(), weight[e].double()
        y[r] = a @ w.t()
        slack[r] = (i + 4) * U32 * (a.abs() @ w.abs().t())
        if bias is not None:
            y[r] += bias[e].double()
            slack[r] += 2 * U32 * bias[e].double().abs()
    return y, slack


def linear_bwd_ref(gys, xs, offsets, weight):
    off = offsets.tolist()
    E, o, i = weight.shape
    z = lambda *s: torch.zeros(s, dtype=torch.float64, device=DEV)
    gx, gw, gb = z(xs.shape[0], i), z(E, o, i), z(E, o)
    sx, sw, sb = z(xs.shape[0], i), z(E, o, i), z(E, o)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        n = off[e + 1] - off[e]
        g, a, w = gys[r].double(), xs[r].double(), weight[e].double()
        gx[r], sx[r] = g @ w, (o + 4) * U32 * (g.abs() @ w.abs())
        gw[e], sw[e] = g.t() @ a, (n + 4) * U32 * (g.abs().t() @ a.abs())
        gb[e], sb[e] = g.sum(0), (n + 4) * U32 * g.abs().sum(0)
    return (gx, gw, gb), (sx, sw, sb)
