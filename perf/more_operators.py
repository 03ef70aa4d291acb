"""Cases of the feature head's router and of its 8-bit operators: experts
chosen from the router's logits with the choices' weights, the experts' counts
and the balance loss; rows kept in 8 bits with a scale for each block of 128;
and the experts' products of such rows -- with their gradients.

A case is computed in one of two forms.  The plain form is elementary torch
operations in 32 bits, rounded once at the end; with `own` set, `run` makes
the library's calls through its binding.  `exact` gives the same outputs from
the definitions in 64 bits.

8-bit rows: q (rows, channels rounded up to 16) in e4m3 and scales (rows, a
byte for every 128 channels, rounded up to 4 bytes) in e8m0; an element is
q * 2^(byte - 127), and a block's byte is the smallest with |x| <= 448 *
2^(byte - 127) for all of the block.
"""

import math

import torch

own = False  # False: the plain form; True: the library's kernels

DEV = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 128


def listed():
    return [
        # one pixel's (or one query point's) choice of experts: latency only
        {"name": "route one token", "kind": "route_fwd", "tokens": 1, "topk": 2, "experts": 8,
         "dtype": "f32", "keep": 1.0, "renormalise": True, "pad": 0},
        # every pixel of a 720p image to two of 16 experts; pixels no splat reaches stay out
        {"name": "route 720p", "kind": "route_fwd", "tokens": 1280 * 720, "topk": 2,
         "experts": 16, "dtype": "f32", "keep": 0.9, "renormalise": True, "pad": 0},
        # the router's gradient in a training step over a batch of pixels, many experts
        {"name": "route grad batch", "kind": "route_bwd", "tokens": 131072, "topk": 4,
         "experts": 64, "dtype": "bf16", "keep": 1.0, "renormalise": True, "pad": 0},
        # odd everything: seven experts in a wider row, weights as they come out of the softmax
        {"name": "route grad odd", "kind": "route_bwd", "tokens": 100003, "topk": 3,
         "experts": 7, "dtype": "f16", "keep": 0.9, "renormalise": False, "pad": 2},
        # a 720p half-precision feature image kept in 8 bits for the backward, and back
        {"name": "pack 720p", "kind": "pack", "rows": 1280 * 720, "channels": 128,
         "dtype": "bf16", "pad": 0},
        # an odd crop with an odd channel count near the raster's 1024-channel limit
        {"name": "pack odd crop", "kind": "pack", "rows": 127 * 129, "channels": 1021,
         "dtype": "f16", "pad": 0},
        # one token's two experts: each product reads its 8-bit weight matrix once
        {"name": "experts 8 bits one token", "kind": "linear_fwd", "tokens": 1, "topk": 2,
         "experts": 8, "in": 256, "out": 1024, "dtype": "bf16", "bias": True, "spread": 0.5,
         "drop": 0.0},
        # an image-sized batch through the experts' first product
        {"name": "experts 8 bits batch", "kind": "linear_fwd", "tokens": 131072, "topk": 2,
         "experts": 16, "in": 512, "out": 1024, "dtype": "bf16", "bias": True, "spread": 0.5,
         "drop": 0.0},
        # a head as wide as the raster's channel limit: bound by the products
        {"name": "experts 8 bits wide", "kind": "linear_fwd", "tokens": 65536, "topk": 1,
         "experts": 4, "in": 1024, "out": 1024, "dtype": "f16", "bias": False, "spread": 0.5,
         "drop": 0.0},
        # answers in 32 bits, odd widths, some pixels dropped
        {"name": "experts 8 bits odd f32", "kind": "linear_fwd", "tokens": 10007, "topk": 2,
         "experts": 6, "in": 259, "out": 131, "dtype": "f32", "bias": True, "spread": 1.0,
         "drop": 0.1},
        # the three gradients in a training step, rows and weights kept in 8 bits
        {"name": "experts 8 bits grad batch", "kind": "linear_bwd", "tokens": 65536, "topk": 2,
         "experts": 16, "in": 512, "out": 1024, "dtype": "bf16", "bias": True, "spread": 0.5,
         "drop": 0.0},
        # the same with gradients in 32 bits and odd widths
        {"name": "experts 8 bits grad odd f32", "kind": "linear_bwd", "tokens": 10007, "topk": 2,
         "experts": 6, "in": 259, "out": 131, "dtype": "f32", "bias": True, "spread": 1.0,
         "drop": 0.1},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["route_fwd", "route_bwd", "pack", "linear_fwd", "linear_bwd"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if kind.startswith("route"):
        experts = _log(rng, 2, 256)
        topk = rng.randint(1, min(experts, 8))
        return {"kind": kind, "tokens": _log(rng, 1, min(1280 * 720, 15_000_000 // experts)),
                "topk": topk, "experts": experts, "dtype": dtype,
                "keep": rng.choice([1.0, 1.0, 0.9, 0.5]),
                # a single weight divided by itself would be 1
                "renormalise": topk > 1 and rng.choice([True, True, False]),
                "pad": rng.choice([0, 0, 3])}
    if kind == "pack":
        channels = _log(rng, 8, 2048)
        return {"kind": kind, "rows": _log(rng, 1, min(1280 * 720, 100_000_000 // channels)),
                "channels": channels, "dtype": dtype, "pad": rng.choice([0, 0, 3, 8])}
    topk = rng.choice([1, 2, 2, 3, 4])
    case = {"kind": kind, "topk": topk, "experts": rng.randint(max(2, topk), 64), "dtype": dtype,
            "spread": rng.choice([0.0, 0.5, 1.0]), "drop": rng.choice([0.0, 0.0, 0.1, 0.5])}
    widths = [_log(rng, 16, 1024) for _ in range(2)]
    if rng.random() < 0.6:  # most heads have widths in whole vectors
        widths = [(w + 7) // 8 * 8 for w in widths]
    most = min(131072, 60_000_000 // max(widths) // topk,
               60_000_000_000 // (widths[0] * widths[1] * topk))
    case.update(tokens=_log(rng, 1, most), bias=rng.choice([True, True, False]))
    case["in"], case["out"] = widths
    return case


# ---- inputs ---------------------------------------------------------------


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _padded(x, pad):
    """x as the last columns of a wider row-major array (a channel slice)."""
    if not pad:
        return x.contiguous()
    wide = torch.empty((x.shape[0], x.shape[1] + pad), dtype=x.dtype, device=x.device)
    wide[:, pad:] = x
    return wide[:, pad:]


def _two_to(byte):
    """2^(byte - 127) as float32."""
    bits = byte.int()
    bits = torch.where(bits > 0, bits << 23, torch.full_like(bits, 1 << 22))
    return bits.view(torch.float32)


def _pack(x):
    """q (rows, channels up to 16) float8_e4m3fn and bytes (rows, blocks up to 4) uint8."""
    rows, ch = x.shape
    blocks = (ch + BLOCK - 1) // BLOCK
    wide = torch.zeros((rows, blocks * BLOCK), device=DEV)
    wide[:, :ch] = x.float()
    wide = wide.reshape(rows, blocks, BLOCK)
    size = torch.where(torch.isfinite(wide), wide.abs(), torch.zeros((), device=DEV))
    bits = size.amax(2).view(torch.int32)
    byte = (bits >> 23) - 8 + ((bits & 0x7fffff) > 0x600000).int()  # 448 = 1.75 * 2^8
    byte = byte.clamp(min=0).to(torch.uint8)
    up = _two_to(254 - byte.int())  # 1 / scale
    q = (wide * up[..., None]).reshape(rows, -1)[:, :(ch + 15) // 16 * 16]
    scales = torch.zeros((rows, (blocks + 3) // 4 * 4), dtype=torch.uint8, device=DEV)
    scales[:, :blocks] = byte
    return q.to(torch.float8_e4m3fn).contiguous(), scales


def _unpack(q, scales, ch):
    """float32 (rows, channels)."""
    each = _two_to(scales).repeat_interleave(BLOCK, 1)[:, :ch]
    return q[:, :ch].float() * each


def _sorted_rows(case, g):
    """offsets (E + 1) of the rows sorted by expert, and how many rows there are."""
    T, k, E = case["tokens"], case["topk"], case["experts"]
    logits = _randn(g, T, E) + case["spread"] * _randn(g, 1, E)
    ids = torch.topk(logits, k, dim=1)[1]
    if case["drop"]:
        gone = torch.rand((T, 1), generator=g, device=DEV) < case["drop"]
        ids = torch.where(gone, torch.full_like(ids, E), ids)
    ranked = torch.sort(ids.reshape(-1))[0]
    return torch.searchsorted(ranked, torch.arange(E + 1, device=DEV)).to(torch.int32)


def prepare(case, seed):
    g = _generator(seed)
    dt = DTYPES[case["dtype"]]
    kind = case["kind"]
    state = {"case": case}
    if kind.startswith("route"):
        T, k, E = case["tokens"], case["topk"], case["experts"]
        # normalised features through a small product: logits around 1, some experts liked more
        state["logits"] = _padded((_randn(g, T, E) + 0.5 * _randn(g, 1, E)).to(dt), case["pad"])
        state["keep"] = None
        if case["keep"] < 1:
            state["keep"] = torch.rand(T, generator=g, device=DEV) < case["keep"]
        if kind == "route_bwd":
            chosen = _route_fwd(state)
            state["ids"], state["counts"] = chosen["ids"], chosen["counts"]
            state["grad_weights"] = _randn(g, T, k)
            state["grad_loss"] = 0.01 * (1 + torch.rand(1, generator=g, device=DEV))
        return state
    if kind == "pack":
        rows, ch = case["rows"], case["channels"]
        # composited features: a scale per pixel, pixels without a splat are 0
        x = _randn(g, rows, ch) * (0.2 + torch.rand((rows, 1), generator=g, device=DEV))
        if rows > 1:
            x *= torch.rand((rows, 1), generator=g, device=DEV) > 0.05
        state["x"] = _padded(x.to(dt), case["pad"])
        return state
    k, m, E = case["in"], case["out"], case["experts"]
    n = case["tokens"] * case["topk"]
    offsets = _sorted_rows(case, g)
    kept = torch.arange(n, device=DEV)[:, None] < offsets[-1]
    state["offsets"] = offsets
    state["xq"], state["xscales"] = _pack(_randn(g, n, k) * kept)
    wq, ws = _pack(_randn(g, E * m, k) / math.sqrt(k))
    state["wq"], state["wscales"] = wq.reshape(E, m, -1), ws.reshape(E, m, -1)
    state["bias"] = (0.1 * _randn(g, E, m)).to(dt) if case["bias"] else None
    # rows of the fullest expert: the plain form lays the experts' rows out to this height
    state["most"] = max(1, int((offsets[1:] - offsets[:-1]).max()))
    if kind == "linear_bwd":
        state["grad_ys"] = (_randn(g, n, m) * kept).to(dt)
    # the types that say what the bytes are
    for name in ("xscales", "wscales"):
        state[name] = state[name].view(torch.float8_e8m0fnu)
    return state


# ---- the plain forms --------------------------------------------------------


def _softmax(x):
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _route_fwd(s):
    case = s["case"]
    T, k, E = case["tokens"], case["topk"], case["experts"]
    x = s["logits"].float()
    p = _softmax(x)
    ids = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :k]
    weights = p.gather(1, ids)
    if case["renormalise"]:
        weights = weights / weights.sum(1, keepdim=True)
    ids = ids.to(torch.int32)
    taking = T
    if s["keep"] is not None:
        keep = s["keep"][:, None]
        ids = torch.where(keep, ids, torch.full_like(ids, -1))
        weights = torch.where(keep, weights, torch.zeros((), device=DEV))
        p = torch.where(keep, p, torch.zeros((), device=DEV))
        taking = s["keep"].sum()
    else:
        taking = torch.full((), T, device=DEV)
    experts = torch.arange(E, device=DEV, dtype=torch.int32)
    pairs = torch.zeros(E, dtype=torch.int64, device=DEV)
    for j in range(k):
        pairs = pairs + (ids[:, j:j + 1] == experts).sum(0)
    share = pairs.float() / pairs.sum().clamp(min=1).float()
    loss = E * (share * p.sum(0) / taking.clamp(min=1).float()).sum()
    counts = torch.cat([pairs, taking.reshape(1)]).to(torch.int32)
    return {"ids": ids, "weights": weights, "counts": counts, "loss": loss.reshape(1)}


def _route_bwd(s):
    case = s["case"]
    E = case["experts"]
    x = s["logits"].float()
    p = _softmax(x)
    pairs, taking = s["counts"][:E].float(), s["counts"][E].float()
    share = pairs / pairs.sum().clamp(min=1)
    per_expert = s["grad_loss"] * E * share / taking.clamp(min=1)
    ids = s["ids"].clamp(min=0).long()
    gw = s["grad_weights"]
    grad = p * (per_expert - (p * per_expert).sum(1, keepdim=True))
    chosen = p.gather(1, ids)
    if case["renormalise"]:
        w = chosen / chosen.sum(1, keepdim=True)
        grad = grad.scatter_add(1, ids, w * (gw - (w * gw).sum(1, keepdim=True)))
    else:
        grad = grad.scatter_add(1, ids, chosen * gw) - p * (chosen * gw).sum(1, keepdim=True)
    grad = torch.where(s["ids"][:, :1] >= 0, grad, torch.zeros((), device=DEV))
    return {"grad_logits": grad.to(s["logits"].dtype)}


def _pack_and_back(s):
    ch = s["case"]["channels"]
    q, scales = _pack(s["x"])
    return {"values": _unpack(q, scales, ch).to(s["x"].dtype),
            "scales": scales[:, :(ch + BLOCK - 1) // BLOCK]}


def _laid_out(rows, offsets, most):
    """Sorted rows as (E, most, width) in 32 bits, zero below each expert's
    last row, with each row's place in it (E * most for rows of no expert)."""
    E = offsets.numel() - 1
    at = torch.arange(rows.shape[0], device=DEV, dtype=torch.int32)
    expert = torch.searchsorted(offsets[1:].contiguous(), at, right=True)
    kept = expert < E
    e = expert.clamp(max=E - 1)
    place = torch.where(kept, e * most + (at - offsets[e]), torch.full_like(e, E * most))
    out = torch.zeros((E * most + 1, rows.shape[1]), device=DEV)
    out[place] = rows.float()
    return out[:E * most].reshape(E, most, -1), place, kept


def _back(block, place, kept, dtype):
    flat = block.reshape(-1, block.shape[2])
    rows = flat[place.clamp(max=flat.shape[0] - 1)]
    return torch.where(kept[:, None], rows, torch.zeros((), device=DEV)).to(dtype)


def _operands(s):
    k = s["case"]["in"]
    xs = _unpack(s["xq"], s["xscales"].view(torch.uint8), k)
    E, m = s["wq"].shape[:2]
    w = _unpack(s["wq"].reshape(E * m, -1), s["wscales"].view(torch.uint8).reshape(E * m, -1), k)
    return xs, w.reshape(E, m, k)


def _linear_fwd(s):
    xs, w = _operands(s)
    x, place, kept = _laid_out(xs, s["offsets"], s["most"])
    y = torch.matmul(x, w.transpose(1, 2))
    if s["bias"] is not None:
        y = y + s["bias"].float()[:, None, :]
    return {"ys": _back(y, place, kept, DTYPES[s["case"]["dtype"]])}


def _linear_bwd(s):
    dt = s["grad_ys"].dtype
    xs, w = _operands(s)
    x, place, kept = _laid_out(xs, s["offsets"], s["most"])
    gy = _laid_out(s["grad_ys"], s["offsets"], s["most"])[0]
    gx = torch.matmul(gy, w)
    gw = torch.matmul(gy.transpose(1, 2), x)
    out = {"grad_xs": _back(gx, place, kept, dt), "grad_weight": gw.to(dt)}
    if s["bias"] is not None:
        out["grad_bias"] = gy.sum(1).to(dt)
    return out


PLAIN = {"route_fwd": _route_fwd, "route_bwd": _route_bwd, "pack": _pack_and_back,
         "linear_fwd": _linear_fwd, "linear_bwd": _linear_bwd}


def _own(s):
    from tile_gaussian_splat_gb300 import binding as gs

    case = s["case"]
    kind = case["kind"]
    if kind == "route_fwd":
        ids, weights, counts, loss = gs.gs_expert_route_fwd(
            s["logits"], case["topk"], keep=s["keep"], renormalise=case["renormalise"])
        return {"ids": ids, "weights": weights, "counts": counts, "loss": loss}
    if kind == "route_bwd":
        return {"grad_logits": gs.gs_expert_route_bwd(
            s["logits"], s["ids"], s["counts"], s["grad_weights"], s["grad_loss"],
            renormalise=case["renormalise"])}
    if kind == "pack":
        ch = case["channels"]
        q, scales = gs.gs_rows_pack8(s["x"])
        return {"values": gs.gs_rows_unpack8(q, scales, ch, s["x"].dtype),
                "scales": scales.view(torch.uint8)[:, :(ch + BLOCK - 1) // BLOCK]}
    if kind == "linear_fwd":
        return {"ys": gs.gs_expert_linear8_fwd(s["xq"], s["xscales"], s["offsets"], s["wq"],
                                               s["wscales"], case["in"], s["bias"],
                                               dtype=DTYPES[case["dtype"]])}
    gx, gw, gb = gs.gs_expert_linear8_bwd(s["grad_ys"], s["xq"], s["xscales"], s["offsets"],
                                          s["wq"], s["wscales"], case["in"],
                                          bias=s["bias"] is not None)
    out = {"grad_xs": gx, "grad_weight": gw}
    if gb is not None:
        out["grad_bias"] = gb
    return out


def run(state):
    return _own(state) if own else PLAIN[state["case"]["kind"]](state)


# ---- what a pass cannot do without --------------------------------------------


def work(case):
    b = SIZES[case["dtype"]]
    kind = case["kind"]
    if kind.startswith("route"):
        T, k, E = case["tokens"], case["topk"], case["experts"]
        kept = case["keep"] * T
        mask = T if case["keep"] < 1 else 0
        if kind == "route_fwd":  # logits in; ids, weights, counts and loss out
            return {"bytes": b * kept * E + mask + 8 * T * k + 4 * E + 8, "flops": 4 * kept * E}
        # logits, ids, grad_weights, counts in; grad_logits out
        return {"bytes": b * kept * E + b * T * E + 4 * T * k + 4 * kept * k + 4 * E + 8,
                "flops": 8 * kept * E}
    if kind == "pack":  # x in, 8 bits and scales out; those in, values out
        n = case["rows"] * case["channels"]
        blocks = case["rows"] * ((case["channels"] + BLOCK - 1) // BLOCK)
        return {"bytes": 2 * n * b + 2 * (n + blocks), "flops": 4 * n}
    T, E = case["tokens"], case["experts"]
    n = T * case["topk"]
    kept = (1 - case["drop"]) * n
    k, m = case["in"], case["out"]
    row = k + (k + BLOCK - 1) // BLOCK  # bytes of an 8-bit row
    used = min(E, math.ceil(kept))  # experts that have a row
    bias = m if case["bias"] else 0
    if kind == "linear_fwd":
        return {"bytes": kept * row + b * n * m + used * (m * row + b * bias) + 4 * E,
                "flops": 2 * kept * k * m}
    return {"bytes": kept * row + b * (kept * m + n * k) + used * m * row +
            b * E * (m * k + bias) + 4 * E, "flops": 4 * kept * k * m}


# ---- the definitions in 64 bits -------------------------------------------------


def _double(power):
    """2^power in 64 bits, to the bit (a power function may be one off)."""
    return ((power.long() + 1023) << 52).view(torch.float64)


def _values(q, scales, ch):
    rows = q.shape[0]
    out = torch.empty((rows, ch), dtype=torch.float64, device=DEV)
    for k0 in range(0, ch, BLOCK):
        size = _double(scales[:, k0 // BLOCK].long() - 127)
        part = slice(k0, min(ch, k0 + BLOCK))
        out[:, part] = q[:, part].double() * size[:, None]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind.startswith("route"):
        T, k, E = case["tokens"], case["topk"], case["experts"]
        x = s["logits"].double().requires_grad_(kind == "route_bwd")
        take = s["keep"] if s["keep"] is not None else torch.ones(T, dtype=torch.bool, device=DEV)
        p = torch.softmax(x, 1)
        if kind == "route_bwd":
            ids = s["ids"].long()
        else:
            left = x.clone()
            number = torch.arange(E, device=DEV).expand(T, E)
            ids = torch.empty((T, k), dtype=torch.int64, device=DEV)
            for j in range(k):
                best = left.max(1, keepdim=True)[0]
                ids[:, j] = torch.where(left == best, number, E).min(1)[0]
                left.scatter_(1, ids[:, j:j + 1], -math.inf)
            ids[~take] = -1
        some = ids.clamp(min=0)
        w = torch.softmax(x.gather(1, some), 1) if case["renormalise"] else p.gather(1, some)
        w = w * take[:, None]
        pairs = torch.bincount(ids[take].reshape(-1), minlength=E)
        taking = int(take.sum())
        loss = (E / max(1, taking)) * ((p * take[:, None]).sum(0) * pairs).sum() / \
            max(1, int(pairs.sum()))
        if kind == "route_bwd":
            ((w * s["grad_weights"].double()).sum() + loss * s["grad_loss"].double()).backward()
            return {"grad_logits": x.grad}
        counts = torch.cat([pairs, torch.tensor([taking], device=DEV)])
        return {"ids": ids.to(torch.int32), "weights": w, "counts": counts.to(torch.int32),
                "loss": loss.reshape(1)}
    if kind == "pack":
        rows, ch = case["rows"], case["channels"]
        values = torch.empty((rows, ch), dtype=torch.float64, device=DEV)
        scales = torch.empty((rows, (ch + BLOCK - 1) // BLOCK), dtype=torch.uint8, device=DEV)
        for k0 in range(0, ch, BLOCK):
            x = s["x"][:, k0:k0 + BLOCK].double()
            most = x.abs().max(1)[0]
            _, power = torch.frexp(most / 448)  # most / 448 = fraction in [1/2, 1) * 2^power
            power = torch.where(448 * _double(power - 1) >= most, power - 1, power)
            power = torch.where(most > 0, power.clamp(min=-127), -127)
            unit = _double(power)[:, None]
            v = x / unit
            _, at = torch.frexp(v)
            step = _double((at - 1).clamp(min=-6) - 3)  # three bits of fraction
            values[:, k0:k0 + BLOCK] = torch.round(v / step) * step * unit
            scales[:, k0 // BLOCK] = (power + 127).to(torch.uint8)
        return {"values": values, "scales": scales}
    off = s["offsets"].tolist()
    n, k, m, E = case["tokens"] * case["topk"], case["in"], case["out"], case["experts"]
    xs = _values(s["xq"], s["xscales"].view(torch.uint8), k)
    matrix = lambda e: _values(s["wq"][e], s["wscales"][e].view(torch.uint8), k)
    if kind == "linear_fwd":
        ys = torch.zeros((n, m), dtype=torch.float64, device=DEV)
        for e in range(E):
            part = xs[off[e]:off[e + 1]] @ matrix(e).t()
            if s["bias"] is not None:
                part += s["bias"][e].double()
            ys[off[e]:off[e + 1]] = part
        return {"ys": ys}
    gx = torch.zeros((n, k), dtype=torch.float64, device=DEV)
    gw = torch.zeros((E, m, k), dtype=torch.float64, device=DEV)
    gb = torch.zeros((E, m), dtype=torch.float64, device=DEV)
    for e in range(E):
        gy = s["grad_ys"][off[e]:off[e + 1]].double()
        gx[off[e]:off[e + 1]] = gy @ matrix(e)
        gw[e] = gy.t() @ xs[off[e]:off[e + 1]]
        gb[e] = gy.sum(0)
    out = {"grad_xs": gx, "grad_weight": gw}
    if s["bias"] is not None:
        out["grad_bias"] = gb
    return out
