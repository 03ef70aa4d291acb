"""Plain 64-bit forms of the router and of the 8-bit rows, and the bounds the
GPU tests hold the kernels to (see head_util for the sums').

Softmax: a difference of two float32 logits is rounded once (2^-24 of its
size, which moves the exponential by that much relatively), the exponential is
within 2 units of the last place, the sum of n of them within (n + 2) * 2^-23
and the division within one unit: together (|difference| + n + 8) * 2^-23.
"""

from __future__ import annotations

import torch

from head_util import DEV, U32

BLOCK = 128


def two_to(power):
    """2^power (int64) in 64 bits, to the bit."""
    return ((power.long() + 1023) << 52).view(torch.float64)


def pack_ref(x):
    """(values in 64 bits, bytes (rows, blocks)): every block's smallest byte
    with |x| <= 448 * 2^(byte - 127), and the nearest e4m3, ties to even."""
    rows, ch = x.shape
    blocks = (ch + BLOCK - 1) // BLOCK
    wide = torch.zeros((rows, blocks * BLOCK), dtype=torch.float64, device=x.device)
    wide[:, :ch] = x.double()
    wide = wide.reshape(rows, blocks, BLOCK)
    finite = torch.isfinite(wide)
    most = torch.where(finite, wide.abs(), 0.0).amax(2)
    byte = torch.zeros_like(most, dtype=torch.int64)
    for b in range(255):  # the smallest that is enough
        byte += (most > 448 * two_to(byte - 127)).long()
    unit = two_to(byte - 127)[..., None]
    v = torch.where(finite, wide, 0.0) / unit
    # steps of e4m3: 2^-9 up to 2^-6, then an eighth of the power of two below
    step = torch.full_like(v, 2.0 ** -9)
    for p in range(-6, 9):
        step = torch.where(v.abs() >= 2.0 ** p, 2.0 ** (p - 3), step)
    q = torch.round(v / step) * step
    values = torch.where(finite, q * unit, float("nan"))
    return values.reshape(rows, -1)[:, :ch], byte


def values_ref(q, scales, ch):
    """What 8-bit rows stand for, in 64 bits."""
    byte = scales.view(torch.uint8).long().repeat_interleave(BLOCK, -1)[..., :ch]
    return q[..., :ch].float().double() * two_to(byte - 127)


def cut(values, dtype):
    """As gs_rows_unpack8 gives them."""
    most = torch.finfo(dtype).max
    return values.clamp(-most, most)


def route_ref(logits, topk, keep, renormalise):
    """(ids, weights, their slack, counts, loss, its slack)."""
    T, E = logits.shape
    x = logits.double().cpu()
    keep = torch.ones(T, dtype=torch.bool) if keep is None else keep.bool().cpu()
    ids = torch.full((T, topk), -1, dtype=torch.int32)
    w = torch.zeros((T, topk), dtype=torch.float64)
    sw = torch.zeros_like(w)
    p_all = torch.zeros((T, E), dtype=torch.float64)
    s_all = torch.zeros_like(p_all)
    for t in range(T):
        row = x[t].tolist()
        order = sorted((e for e in range(E) if row[e] != float("-inf")),
                       key=lambda e: (-float("inf") if row[e] != row[e] else -row[e],
                                      0 if row[e] != row[e] else 1, e))
        if not keep[t] or not order:
            continue
        keep_here = order[:topk]
        top = row[order[0]]
        d = (x[t] - top)
        e = torch.exp(d)
        p = e / e.sum()
        rel = (torch.where(torch.isfinite(d), d.abs(), torch.zeros(())) + E + 8) * U32
        p_all[t], s_all[t] = p, p * (rel + rel.max())
        chosen = torch.tensor(keep_here)
        ids[t, :len(keep_here)] = chosen.int()
        mine = p[chosen] / p[chosen].sum() if renormalise else p[chosen]
        w[t, :len(keep_here)] = mine
        sw[t, :len(keep_here)] = mine * (rel[chosen] + rel[chosen].max() + rel.max())
    took = ids[:, 0] >= 0
    pairs = torch.bincount(ids[ids >= 0].long(), minlength=E)
    taking = int(took.sum())
    loss = slack = 0.0
    if taking:
        share = pairs.double() / pairs.sum()
        loss = float(E * (share * p_all.sum(0) / taking).sum())
        # sums over the tokens in float32, then over the experts
        slack = float(E * (share * s_all.sum(0) / taking).sum()) + loss * (T + E + 16) * U32
    counts = torch.cat([pairs, torch.tensor([taking])]).int()
    return (ids.to(DEV), w.to(DEV), sw.to(DEV), counts.to(DEV), loss, slack)


def route_bwd_ref(logits, ids, counts, gw, gl, renormalise):
    """(grad_logits, slack), by the formula."""
    T, E = logits.shape
    k = ids.shape[1]
    took = (ids[:, 0] >= 0)
    x = torch.where(took[:, None], logits.double(), 0.0)
    top = x.amax(1, keepdim=True)
    d = x - top
    e = torch.exp(d)
    p = e / e.sum(1, keepdim=True)
    size = torch.where(torch.isfinite(d), d.abs(), 0.0)
    rel = (size + E + 8) * U32
    rel = rel + rel.amax(1, keepdim=True)
    h = torch.zeros(E, dtype=torch.float64, device=logits.device)
    if gl is not None:
        pairs = counts[:E].double()
        h = gl.double() * E * pairs / pairs.sum().clamp(min=1) / counts[E].double().clamp(min=1)
    ph = (p * h).sum(1, keepdim=True)
    grad = p * (h - ph)
    # every factor and sum again, each within rel, the sum's terms E more
    slack = p * (h.abs() + (p * h.abs()).sum(1, keepdim=True)) * (3 * rel + (E + 8) * U32)
    if gw is not None:
        have = ids >= 0
        at = ids.clamp(min=0).long()
        chosen = torch.where(have, p.gather(1, at), 0.0)
        r = torch.where(have, rel.gather(1, at), 0.0).amax(1, keepdim=True) + rel.amax(1, keepdim=True)
        g = torch.where(have, gw.double(), 0.0)
        if renormalise:
            w = chosen / chosen.sum(1, keepdim=True).clamp(min=1e-300)
            mean = (w * g).sum(1, keepdim=True)
            add = w * (g - mean)
            s = w * (g.abs() + (w * g.abs()).sum(1, keepdim=True)) * (3 * r + (k + 8) * U32)
        else:
            add = chosen * g
            s = add.abs() * (3 * r + 8 * U32)
            down = add.sum(1, keepdim=True)
            grad = grad - p * down
            slack = slack + p * add.abs().sum(1, keepdim=True) * (3 * r + (k + 8) * U32)
        grad = grad.scatter_add(1, at, add)
        slack = slack.scatter_add(1, at, s)
    none = torch.zeros((), dtype=torch.float64, device=logits.device)
    return torch.where(took[:, None], grad, none), torch.where(took[:, None], slack, none)
