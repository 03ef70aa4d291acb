"""Cases of the feature-head operators: layer norm over the channels of a
rendered feature image, tokens (pixels) sorted by expert and back with their
weights, and the experts' products -- each forward and backward.

A case is computed in one of two forms.  The plain form is elementary torch
operations in 32 bits, rounded once at the end; with `own` set, `run` makes
the library's calls through its binding.  `exact` gives the same outputs from
the definitions in 64 bits.
"""

import math

import torch

own = False  # False: the plain form; True: the library's kernels

DEV = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5


def listed():
    return [
        # one pixel's (or one query point's) features through the head: latency only
        {"name": "norm one pixel", "kind": "norm_fwd", "rows": 1, "channels": 64, "dtype": "f32",
         "param": "f32", "pad": 0},
        # a full-HD feature render, 64 feature channels behind 3 colour channels of one
        # (H, W, 67) image: the norm reads the channel slice in place
        {"name": "norm full HD slice", "kind": "norm_fwd", "rows": 1920 * 1080, "channels": 64,
         "dtype": "f32", "param": "f32", "pad": 3},
        # the training step of a 720p half-precision feature image
        {"name": "norm grad 720p", "kind": "norm_bwd", "rows": 1280 * 720, "channels": 128,
         "dtype": "bf16", "param": "f32", "pad": 0},
        # an odd crop with an odd channel count near the raster's 1024-channel limit
        {"name": "norm grad odd crop", "kind": "norm_bwd", "rows": 127 * 129, "channels": 1021,
         "dtype": "f16", "param": "f16", "pad": 0},
        # one token to its two experts: the serving call, latency only
        {"name": "dispatch one token", "kind": "dispatch", "tokens": 1, "topk": 2, "experts": 8,
         "channels": 256, "dtype": "bf16", "spread": 0.5, "drop": 0.0, "pad": 0},
        # every pixel of a 720p image to two of 16 experts; pixels no splat reaches are dropped
        {"name": "dispatch 720p", "kind": "dispatch", "tokens": 1280 * 720, "topk": 2,
         "experts": 16, "channels": 64, "dtype": "f32", "spread": 0.5, "drop": 0.1, "pad": 0},
        # odd everything: a ragged batch of pixels, three experts each of seven
        {"name": "combine odd", "kind": "combine", "tokens": 100003, "topk": 3, "experts": 7,
         "channels": 131, "dtype": "f16", "weighted": True, "spread": 1.0, "drop": 0.1, "pad": 0},
        # the combine's backward in a training step over a batch of pixel features
        {"name": "combine grad batch", "kind": "combine_bwd", "tokens": 131072, "topk": 2,
         "experts": 32, "channels": 512, "dtype": "bf16", "spread": 0.5, "drop": 0.0, "pad": 0},
        # one token's two experts: each product reads its weight matrix once
        {"name": "experts one token", "kind": "linear_fwd", "tokens": 1, "topk": 2, "experts": 8,
         "in": 256, "out": 1024, "dtype": "bf16", "bias": True, "spread": 0.5, "drop": 0.0},
        # a prompt-sized or image-sized batch through the experts' first product
        {"name": "experts batch", "kind": "linear_fwd", "tokens": 131072, "topk": 2,
         "experts": 16, "in": 512, "out": 1024, "dtype": "bf16", "bias": True, "spread": 0.5,
         "drop": 0.0},
        # the same product's three gradients in a training step
        {"name": "experts grad batch", "kind": "linear_bwd", "tokens": 65536, "topk": 2,
         "experts": 16, "in": 512, "out": 1024, "dtype": "bf16", "bias": True, "spread": 0.5,
         "drop": 0.0},
        # a head kept in 32 bits with odd widths, some pixels dropped
        {"name": "experts odd f32", "kind": "linear_fwd", "tokens": 10007, "topk": 2,
         "experts": 6, "in": 259, "out": 131, "dtype": "f32", "bias": True, "spread": 1.0,
         "drop": 0.1},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["norm_fwd", "norm_bwd", "dispatch", "combine", "combine_bwd",
                       "linear_fwd", "linear_bwd"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if kind.startswith("norm"):
        channels = _log(rng, 8, 1024)
        rows = _log(rng, 1, min(1920 * 1080, 100_000_000 // channels))
        return {"kind": kind, "rows": rows, "channels": channels, "dtype": dtype,
                "param": rng.choice(["f32", dtype]), "pad": rng.choice([0, 0, 3, 8])}
    topk = rng.choice([1, 2, 2, 3, 4])
    case = {"kind": kind, "topk": topk, "experts": rng.randint(max(2, topk), 64), "dtype": dtype,
            "spread": rng.choice([0.0, 0.5, 1.0]), "drop": rng.choice([0.0, 0.0, 0.1, 0.5])}
    if not kind.startswith("linear"):
        channels = _log(rng, 8, 1024)
        tokens = _log(rng, 1, min(1280 * 720, 60_000_000 // (topk * channels)))
        case.update(tokens=tokens, channels=channels, pad=rng.choice([0, 0, 3]))
        if kind == "combine":
            case["weighted"] = rng.choice([True, True, False])
        return case
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


def _route(case, g):
    """Router output: topk distinct experts per token with softmax weights;
    some experts are liked more than others, dropped tokens have -1."""
    T, k, E = case["tokens"], case["topk"], case["experts"]
    logits = _randn(g, T, E) + case["spread"] * _randn(g, 1, E)
    top, ids = torch.topk(logits, k, dim=1)
    weights = torch.softmax(top, 1)
    if case["drop"]:
        gone = torch.rand((T, 1), generator=g, device=DEV) < case["drop"]
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    return ids.to(torch.int32).contiguous(), weights.contiguous()


def _sorted_by_expert(ids, experts):
    """offsets (E+1), order (T*k) and slots (T, k) of the stable sort by expert."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < experts), flat, torch.full_like(flat, experts))
    ranked, order = torch.sort(key, stable=True)
    bounds = torch.arange(experts + 1, device=ids.device)
    offsets = torch.searchsorted(ranked, bounds).to(torch.int32)
    kept = ranked < experts
    slots = torch.empty(n, dtype=torch.int32, device=ids.device)
    at = torch.arange(n, dtype=torch.int32, device=ids.device)
    slots[order] = torch.where(kept, at, torch.full_like(at, -1))
    order = torch.where(kept, order, torch.full_like(order, -1)).to(torch.int32)
    return offsets, order, slots.reshape(ids.shape)


def prepare(case, seed):
    g = _generator(seed)
    dt = DTYPES[case["dtype"]]
    kind = case["kind"]
    state = {"case": case}
    if kind.startswith("norm"):
        rows, ch = case["rows"], case["channels"]
        # composited features: an offset and a scale per pixel, pixels without a splat are 0
        x = _randn(g, rows, ch) * (0.2 + torch.rand((rows, 1), generator=g, device=DEV))
        x += 0.5 * _randn(g, rows, 1)
        if rows > 1:
            x *= torch.rand((rows, 1), generator=g, device=DEV) > 0.05
        p = DTYPES[case["param"]]
        state["x"] = _padded(x.to(dt), case["pad"])
        state["weight"] = (1 + 0.1 * _randn(g, ch)).to(p)
        state["bias"] = (0.1 * _randn(g, ch)).to(p)
        if kind == "norm_bwd":
            state["grad_y"] = _randn(g, rows, ch).to(dt)
            xf = state["x"].float()
            mean = xf.mean(1)
            var = (xf - mean[:, None]).square().mean(1)
            state["mean"], state["rstd"] = mean.contiguous(), torch.rsqrt(var + EPS).contiguous()
        return state
    ids, weights = _route(case, g)
    n = ids.numel()
    offsets, order, slots = _sorted_by_expert(ids, case["experts"])
    if kind == "dispatch":
        state["ids"] = ids
        state["x"] = _padded(_randn(g, case["tokens"], case["channels"]).to(dt), case["pad"])
        return state
    state["offsets"] = offsets
    if kind.startswith("combine"):
        state["slots"] = slots
        ys = _randn(g, n, case["channels"])
        ys *= (order >= 0)[:, None]
        state["ys"] = ys.to(dt)
        state["weights"] = weights if case.get("weighted", True) else None
        if kind == "combine_bwd":
            state["grad_y"] = _padded(_randn(g, case["tokens"], case["channels"]).to(dt),
                                      case["pad"])
        return state
    k, m, E = case["in"], case["out"], case["experts"]
    xs = _randn(g, n, k)
    xs *= (order >= 0)[:, None]
    state["xs"] = xs.to(dt)
    state["weight"] = (_randn(g, E, m, k) / math.sqrt(k)).to(dt)
    state["bias"] = (0.1 * _randn(g, E, m)).to(dt) if case["bias"] else None
    # rows of the fullest expert: the plain form lays the experts' rows out to this height
    state["most"] = max(1, int((offsets[1:] - offsets[:-1]).max()))
    if kind == "linear_bwd":
        gys = _randn(g, n, m)
        gys *= (order >= 0)[:, None]
        state["grad_ys"] = gys.to(dt)
    return state


# ---- the plain forms --------------------------------------------------------


def _norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = torch.rsqrt((d * d).mean(1, keepdim=True) + EPS)
    y = d * rstd * s["weight"].float() + s["bias"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _norm_bwd(s):
    gy = s["grad_y"].float()
    rstd = s["rstd"][:, None]
    xhat = (s["x"].float() - s["mean"][:, None]) * rstd
    g = gy * s["weight"].float()
    gx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    p = s["weight"].dtype
    return {"grad_x": gx.to(s["x"].dtype), "grad_weight": (gy * xhat).sum(0).to(p),
            "grad_bias": gy.sum(0).to(p)}


def _dispatch(s):
    case = s["case"]
    offsets, order, slots = _sorted_by_expert(s["ids"], case["experts"])
    kept = (order >= 0)[:, None]
    token = order.clamp(min=0).long() // case["topk"]
    xs = torch.where(kept, s["x"][token], torch.zeros((), dtype=s["x"].dtype, device=DEV))
    return {"offsets": offsets, "order": order, "slots": slots, "xs": xs}


def _taken(s):
    """ys by token and choice, in 32 bits, 0 where the choice was dropped."""
    slots = s["slots"].long()
    rows = s["ys"][slots.clamp(min=0)].float()
    return torch.where((slots >= 0)[..., None], rows, torch.zeros((), device=DEV))


def _combine(s):
    rows = _taken(s)
    if s["weights"] is not None:
        rows = rows * s["weights"][..., None]
    return {"y": rows.sum(1).to(s["ys"].dtype)}


def _combine_bwd(s):
    gy = s["grad_y"].float()[:, None, :]
    grad_w = (_taken(s) * gy).sum(2)
    flat = s["slots"].reshape(-1).long()
    n = flat.numel()
    rows = (gy * s["weights"][..., None]).reshape(n, -1).to(s["ys"].dtype)
    spare = torch.zeros((n + 1, rows.shape[1]), dtype=rows.dtype, device=DEV)
    spare[torch.where(flat >= 0, flat, torch.full_like(flat, n))] = rows
    return {"grad_ys": spare[:n], "grad_weights": grad_w}


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


def _linear_fwd(s):
    x, place, kept = _laid_out(s["xs"], s["offsets"], s["most"])
    y = torch.matmul(x, s["weight"].float().transpose(1, 2))
    if s["bias"] is not None:
        y = y + s["bias"].float()[:, None, :]
    return {"ys": _back(y, place, kept, s["xs"].dtype)}


def _linear_bwd(s):
    dt = s["xs"].dtype
    x, place, kept = _laid_out(s["xs"], s["offsets"], s["most"])
    gy = _laid_out(s["grad_ys"], s["offsets"], s["most"])[0]
    gx = torch.matmul(gy, s["weight"].float())
    gw = torch.matmul(gy.transpose(1, 2), x)
    out = {"grad_xs": _back(gx, place, kept, dt), "grad_weight": gw.to(dt)}
    if s["bias"] is not None:
        out["grad_bias"] = gy.sum(1).to(dt)
    return out


PLAIN = {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "dispatch": _dispatch,
         "combine": _combine, "combine_bwd": _combine_bwd, "linear_fwd": _linear_fwd,
         "linear_bwd": _linear_bwd}


def _own(s):
    from tile_gaussian_splat_gb300 import binding as gs

    case = s["case"]
    kind = case["kind"]
    if kind == "norm_fwd":
        y, mean, rstd = gs.gs_layer_norm_fwd(s["x"], s["weight"], s["bias"], EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if kind == "norm_bwd":
        gx, gw, gb = gs.gs_layer_norm_bwd(s["grad_y"], s["x"], s["weight"], s["mean"], s["rstd"])
        return {"grad_x": gx, "grad_weight": gw, "grad_bias": gb}
    if kind == "dispatch":
        offsets, order, slots = gs.gs_expert_sort(s["ids"], case["experts"])
        return {"offsets": offsets, "order": order, "slots": slots,
                "xs": gs.gs_expert_dispatch(s["x"], slots, offsets)}
    if kind == "combine":
        return {"y": gs.gs_expert_combine(s["ys"], s["slots"], s["weights"])}
    if kind == "combine_bwd":
        gys, gw = gs.gs_expert_combine_bwd(s["grad_y"], s["ys"], s["slots"], s["weights"],
                                           s["offsets"])
        return {"grad_ys": gys, "grad_weights": gw}
    if kind == "linear_fwd":
        return {"ys": gs.gs_expert_linear_fwd(s["xs"], s["offsets"], s["weight"], s["bias"])}
    gx, gw, gb = gs.gs_expert_linear_bwd(s["grad_ys"], s["xs"], s["offsets"], s["weight"],
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
    if kind.startswith("norm"):
        n, ch = case["rows"] * case["channels"], case["channels"]
        p = SIZES[case["param"]] * ch
        if kind == "norm_fwd":  # x in, y out, two statistics a row, weight and bias
            return {"bytes": 2 * n * b + 8 * case["rows"] + 2 * p, "flops": 8 * n}
        # x, grad_y in, grad_x out, the statistics, weight in and two gradients out
        return {"bytes": 3 * n * b + 8 * case["rows"] + 3 * p, "flops": 16 * n}
    T, E = case["tokens"], case["experts"]
    n = T * case["topk"]
    kept = (1 - case["drop"]) * n
    if kind == "dispatch":  # ids, x in; offsets, order, slots and the sorted rows out
        ch = case["channels"]
        return {"bytes": 12 * n + 4 * E + (1 - case["drop"]) * T * ch * b + n * ch * b,
                "flops": 0}
    if kind == "combine":
        ch = case["channels"]
        w = 4 * n if case["weighted"] else 0
        return {"bytes": 4 * n + w + kept * ch * b + T * ch * b, "flops": 2 * kept * ch}
    if kind == "combine_bwd":  # grad_y, ys, slots, weights in; grad_ys, grad_weights out
        ch = case["channels"]
        return {"bytes": 12 * n + (1 - case["drop"]) * T * ch * b + kept * ch * b + n * ch * b,
                "flops": 3 * kept * ch}
    k, m = case["in"], case["out"]
    used = min(E, math.ceil(kept))  # experts that have a row
    bias = m if case["bias"] else 0
    if kind == "linear_fwd":
        return {"bytes": b * (kept * k + n * m + used * (m * k + bias)) + 4 * E,
                "flops": 2 * kept * k * m}
    return {"bytes": b * (kept * (k + m) + n * k + used * m * k + E * (m * k + bias)) + 4 * E,
            "flops": 4 * kept * k * m}


# ---- the definitions in 64 bits -------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind.startswith("norm"):
        x = s["x"].double()
        c = case["channels"]
        w = s["weight"].double()
        if kind == "norm_fwd":
            mu = x.sum(dim=1) / c
            var = ((x - mu.unsqueeze(1)) ** 2).sum(dim=1) / c
            inv = 1.0 / torch.sqrt(var + EPS)
            y = (x - mu.unsqueeze(1)) * inv.unsqueeze(1) * w + s["bias"].double()
            return {"y": y, "mean": mu, "rstd": inv}
        # given the statistics that came with the call
        inv = s["rstd"].double().unsqueeze(1)
        n = (x - s["mean"].double().unsqueeze(1)) * inv
        gy = s["grad_y"].double()
        gn = gy * w
        gx = inv * (gn - (gn.sum(1, keepdim=True) + n * (gn * n).sum(1, keepdim=True)) / c)
        return {"grad_x": gx, "grad_weight": torch.einsum("rc,rc->c", gy, n),
                "grad_bias": gy.sum(0)}
    if kind == "dispatch":
        ids = s["ids"].reshape(-1).tolist()
        if len(ids) > 4_000_000:
            return None
        lists = [[] for _ in range(case["experts"])]
        for i, e in enumerate(ids):
            if e >= 0:
                lists[e].append(i)
        order, offsets = [], [0]
        for rows in lists:
            order += rows
            offsets.append(len(order))
        slots = [-1] * len(ids)
        for at, i in enumerate(order):
            slots[i] = at
        xs = torch.zeros((len(ids), case["channels"]), dtype=torch.float64, device=DEV)
        token = torch.tensor([i // case["topk"] for i in order], dtype=torch.int64, device=DEV)
        xs[:len(order)] = s["x"].double()[token]
        order += [-1] * (len(ids) - len(order))
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
        return {"offsets": ints(offsets), "order": ints(order),
                "slots": ints(slots).reshape(s["ids"].shape), "xs": xs}
    if kind.startswith("combine"):
        T, k, ch = case["tokens"], case["topk"], case["channels"]
        ys = s["ys"].double()
        y = torch.zeros((T, ch), dtype=torch.float64, device=DEV)
        grad_ys = torch.zeros_like(ys)
        grad_w = torch.zeros((T, k), dtype=torch.float64, device=DEV)
        for j in range(k):
            rows = torch.nonzero(s["slots"][:, j] >= 0)[:, 0]
            at = s["slots"][rows, j].long()
            w = s["weights"][rows, j].double() if s["weights"] is not None else \
                torch.ones(rows.numel(), dtype=torch.float64, device=DEV)
            if kind == "combine":
                y[rows] += w[:, None] * ys[at]
            else:
                gy = s["grad_y"].double()[rows]
                grad_ys[at] = w[:, None] * gy
                grad_w[rows, j] = torch.einsum("rc,rc->r", gy, ys[at])
        return {"y": y} if kind == "combine" else {"grad_ys": grad_ys, "grad_weights": grad_w}
    off = s["offsets"].tolist()
    n, k, m, E = case["tokens"] * case["topk"], case["in"], case["out"], case["experts"]
    if kind == "linear_fwd":
        ys = torch.zeros((n, m), dtype=torch.float64, device=DEV)
        for e in range(E):
            part = s["xs"][off[e]:off[e + 1]].double() @ s["weight"][e].double().t()
            if s["bias"] is not None:
                part += s["bias"][e].double()
            ys[off[e]:off[e + 1]] = part
        return {"ys": ys}
    gx = torch.zeros((n, k), dtype=torch.float64, device=DEV)
    gw = torch.zeros((E, m, k), dtype=torch.float64, device=DEV)
    gb = torch.zeros((E, m), dtype=torch.float64, device=DEV)
    for e in range(E):
        gy = s["grad_ys"][off[e]:off[e + 1]].double()
        gx[off[e]:off[e + 1]] = gy @ s["weight"][e].double()
        gw[e] = gy.t() @ s["xs"][off[e]:off[e + 1]].double()
        gb[e] = gy.sum(0)
    out = {"grad_xs": gx, "grad_weight": gw}
    if s["bias"] is not None:
        out["grad_bias"] = gb
    return out
