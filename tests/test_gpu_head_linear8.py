"""The experts' products of 8-bit rows (gs_expert_linear8_fwd / _bwd) against
their 64-bit form.

Every product of two 8-bit elements is exact in float32, so a sum of n of them
is off by at most the bound of head_util's sums; the gradients' products are
those of gs_expert_linear_bwd."""

import pytest
import torch

from head8_util import cut, values_ref
from head_util import (DEV, TYPES, check, gen, linear_bwd_ref, linear_ref, randn, routed)
from tile_gaussian_splat_gb300 import binding as gs

pytestmark = pytest.mark.gpu

# (tokens, topk, experts, in, out)
SHAPES = [(1, 1, 1, 1, 1), (1, 2, 8, 256, 1024), (3, 2, 4, 16, 16), (8, 2, 3, 131, 77),
          (20, 1, 2, 128, 128), (100, 2, 4, 64, 192), (333, 2, 5, 129, 193), (500, 3, 7, 48, 24),
          (700, 2, 3, 512, 384), (257, 1, 2, 640, 1000), (1500, 2, 40, 200, 72),
          (2000, 1, 1, 1030, 260), (4000, 2, 6, 259, 131), (129, 1, 1, 2048, 64),
          (20000, 2, 4, 300, 200), (6000, 2, 16, 128, 1000), (1300, 1, 2, 4200, 9000),
          (30000, 1, 300, 128, 256), (9000, 1, 3, 700, 800), (8000, 1, 2, 512, 520),
          (12000, 1, 900, 1100, 200), (700, 2, 3, 202, 130), (20000, 2, 2, 66, 250)]


def _packed(seed, rows, E, i, o, kept):
    g = gen(seed)
    x = randn(g, rows, i) * torch.exp(randn(g, rows, 1))
    x[kept:] = 0
    w = randn(g, E * o, i) * torch.exp(randn(g, E * o, 1)) / i ** 0.5
    xq, xs = gs.gs_rows_pack8(x)
    wq, ws = gs.gs_rows_pack8(w)
    return xq, xs, wq.reshape(E, o, -1), ws.reshape(E, o, -1)


def _values(p, i, dtype=None):
    out = values_ref(p[0], p[1], i), values_ref(p[2], p[3], i)
    return out if dtype is None else tuple(cut(v, dtype).to(dtype).double() for v in out)


def _check_fwd(p, offsets, i, bias, dtype):
    st = gs.new_status(DEV)
    ys = gs.gs_expert_linear8_fwd(p[0], p[1], offsets, p[2], p[3], i, bias, dtype=dtype,
                                  d_status=st)
    gs.check_status(st)
    x, w = _values(p, i)
    ref, slack = linear_ref(x, offsets, w, bias)
    check(ys, ref, slack, "ys")
    return ys


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("tokens,topk,experts,i,o", SHAPES)
def test_forward_and_backward(tokens, topk, experts, i, o, dtype):
    seed = tokens + 7 * i + o
    _, offsets, _, _ = routed(seed, tokens, topk, experts)
    R = tokens * topk
    p = _packed(seed, R, experts, i, o, int(offsets[-1]))
    g = gen(seed + 1)
    for bias in (None, randn(g, experts, o, dtype=dtype)):
        _check_fwd(p, offsets, i, bias, dtype)
    gys = randn(g, R, o, dtype=dtype)
    st = gs.new_status(DEV)
    grads = gs.gs_expert_linear8_bwd(gys, p[0], p[1], offsets, p[2], p[3], i, d_status=st)
    gs.check_status(st)
    # float16 gradients take the values as float16
    x, w = _values(p, i, torch.float16 if dtype == torch.float16 else None)
    refs, slacks = linear_bwd_ref(gys, x, offsets, w)
    for got, ref, slack, what in zip(grads, refs, slacks, ("grad_xs", "grad_weight", "grad_bias")):
        check(got, ref, slack, what)
    none, gw, no = gs.gs_expert_linear8_bwd(gys, p[0], p[1], offsets, p[2], p[3], i, bias=False,
                                            input=False)
    assert none is None and no is None and torch.equal(gw, grads[1])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_experts_without_rows_and_rows_without_experts(dtype):
    _, offsets, _, _ = routed(3, 600, 2, 9, drop=0.4, to=[2, 3, 7])
    kept = int(offsets[-1])
    p = _packed(3, 1200, 9, 160, 144, 1200)  # the rows behind the last expert's hold numbers
    ys = _check_fwd(p, offsets, 160, None, dtype)
    assert not bool(ys[kept:].any())
    # nor does a NaN there reach a result
    raw = p[0].view(torch.uint8)
    raw[kept:] = 0x7f
    assert torch.equal(ys, gs.gs_expert_linear8_fwd(p[0], p[1], offsets, p[2], p[3], 160,
                                                    dtype=dtype))
    gys = randn(gen(4), 1200, 144, dtype=dtype)
    gys[kept:] = float("nan")
    gx, gw, gb = gs.gs_expert_linear8_bwd(gys, p[0], p[1], offsets, p[2], p[3], 160)
    assert not bool(gx[kept:].any())
    for e in (0, 1, 4, 5, 6, 8):
        assert not bool(gw[e].any()) and not bool(gb[e].any())
    x, w = _values(p, 160, torch.float16 if dtype == torch.float16 else None)
    refs, slacks = linear_bwd_ref(gys[:kept], x[:kept], offsets, w)
    for got, ref, slack in zip((gx[:kept], gw, gb), refs, slacks):
        check(got, ref, slack, "gradients")


def test_scales_far_apart():
    """Blocks of a row whose powers of two differ by far more than the
    elements' own range."""
    g = gen(21)
    E, R, i, o = 2, 400, 700, 96
    powers = torch.tensor([-30, 20, 0, -5, 11, 3], device=DEV)
    each = torch.exp2(powers.float()).repeat_interleave(128)[:i]
    x, w = randn(g, R, i) * each, randn(g, E * o, i) * each.flip(0)
    p = (*gs.gs_rows_pack8(x), *(t.reshape(E, o, -1) for t in gs.gs_rows_pack8(w)))
    offsets = torch.tensor([0, 150, 400], dtype=torch.int32, device=DEV)
    for dtype in (torch.float32, torch.bfloat16):
        _check_fwd(p, offsets, i, None, dtype)


@pytest.mark.parametrize("i", [512, 1700, 4352])
def test_every_block_of_channels_meets_its_own_powers(i):
    """Rows that two blocks of threads share, every power another one: a word of
    powers that came too late would leave its buffer's last ones.  Blocks of one
    value, so that all sums are whole multiples of 2^-4 below 2^17: exact."""
    g = gen(60 + i)
    E, R, o, n = 3, 40000, 520, (i + 127) // 128
    power = lambda rows: torch.randint(-2, 3, (rows, n), generator=g, device=DEV)
    spread = lambda p: torch.exp2(p.float()).repeat_interleave(128, 1)[:, :i]
    a, b = power(R), power(E * o)
    p = (*gs.gs_rows_pack8(spread(a)),
         *(t.reshape(E, o, -1) for t in gs.gs_rows_pack8(spread(b))))
    offsets = torch.tensor([0, 13001, 26002, R], dtype=torch.int32, device=DEV)
    wide = torch.full((n,), 128.0, dtype=torch.float64, device=DEV)
    wide[-1] = i - 128 * (n - 1)
    x, w = torch.exp2(a.double()) * wide, torch.exp2(b.double()).reshape(E, o, n)
    want = torch.cat([x[lo:hi] @ w[e].t() for e, (lo, hi) in
                      enumerate(zip(offsets.tolist(), offsets.tolist()[1:]))])
    for _ in range(5):
        ys = gs.gs_expert_linear8_fwd(p[0], p[1], offsets, p[2], p[3], i, dtype=torch.float32)
        assert torch.equal(ys.double(), want)


@pytest.mark.parametrize("rows,i,o", [(9, 300, 40), (700, 400, 96), (30000, 512, 520)])
@pytest.mark.parametrize("high,low", [(18, 18), (-20, -20), (18, -4), (100, 100), (-110, -120),
                                      (18, -20), (60, -60)])
def test_float16_gradients_of_values_beyond_float16(high, low, rows, i, o):
    """Blocks around 2^high and 2^low, gradients that bring the sums back into
    float16 where it has such: each value counts exactly, or to within 2^-39 of
    the largest (the lowest bytes' of all)."""
    g = gen(70 + high + low)
    E = 4
    offsets = torch.tensor([0, rows // 3, rows // 3, rows - 2, rows - 1], dtype=torch.int32,
                           device=DEV)
    at = torch.arange(i, device=DEV) // 128 % 2
    each = torch.exp2(torch.where(at == 0, high, low).double()).float()
    p = (*gs.gs_rows_pack8(randn(g, rows, i) * each),
         *(t.reshape(E, o, -1) for t in gs.gs_rows_pack8(randn(g, E * o, i) * each)))
    size = 2.0 ** max(min(-high, 8), -12)
    gys = (randn(g, rows, o) * size).half()
    run = lambda: gs.gs_expert_linear8_bwd(gys, p[0], p[1], offsets, p[2], p[3], i)
    grads = run()
    x, w = _values(p, i)
    refs, slacks = linear_bwd_ref(gys, x, offsets, w)
    count = gys.double().abs()
    beyond = (2.0 ** -39 * w.abs().max() * count.sum(1, keepdim=True),
              2.0 ** -39 * x.abs().max() * torch.stack(
                  [count[a:b].sum(0) for a, b in zip(offsets.tolist(), offsets.tolist()[1:])]
              )[..., None], 0.0)
    most = torch.finfo(torch.float16).max
    for got, ref, slack, more in zip(grads, refs, slacks, beyond):
        held = ref.abs() + slack + more <= most
        none = torch.zeros((), dtype=torch.float64, device=DEV)
        check(torch.where(held, got, 0), torch.where(held, ref, none),
              torch.where(held, slack + more, none), "gradients")
        over = ref.abs() - slack - more >= 2 * most
        assert bool((got[over].double() == ref[over].sign() * float("inf")).all())
    # nor do powers count that no expert uses, nor what stands for no number
    p[1].view(torch.uint8)[rows - 1:] = 254
    p[3].view(torch.uint8)[1] = 254
    p[3].view(torch.uint8)[..., (i + 127) // 128:] = 254
    assert all(torch.equal(a, b) for a, b in zip(run(), grads))
    p[3].view(torch.uint8)[0, 3, 0] = 255
    assert torch.equal(run()[1], grads[1]) and torch.equal(run()[0][rows // 3:],
                                                           grads[0][rows // 3:])


def test_float16_gradients_captured_and_at_once():
    """The powers that the operands have in common are of the call's own data:
    of a replay's, and of either of two streams'."""
    _, offsets, _, _ = routed(90, 3000, 2, 8)
    a, b = _packed(90, 6000, 8, 256, 320, 6000), _packed(91, 6000, 8, 256, 320, 6000)
    for t in (b[1], b[3]):
        t.view(torch.uint8).sub_(40)
    gys = randn(gen(90), 6000, 320, dtype=torch.float16)
    run = lambda r: gs.gs_expert_linear8_bwd(gys, r[0], r[1], offsets, r[2], r[3], 256)
    want = run(a), run(b)
    assert not torch.equal(want[0][1], want[1][1])
    p = tuple(t.clone() for t in a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(p)
    for r, w in ((b, want[1]), (a, want[0]), (b, want[1])):
        for t, u in zip(p, r):
            t.view(torch.uint8).copy_(u.view(torch.uint8))
        graph.replay()
        assert all(torch.equal(x, y) for x, y in zip(out, w))
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s, r in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                got.append(run(r))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(g, want[i % 2]))


@pytest.mark.parametrize("rows", [5, 700])
def test_values_at_the_end_of_float32(rows):
    """float32's largest value is kept as 2^128; times small weights it is finite."""
    g = gen(50)
    x, w = randn(g, rows, 200), randn(g, 96, 200) * 2.0 ** -30
    x[1, 3], x[2, 150], x[3, 7] = 3.4e38, -torch.finfo(torch.float32).max, 2.0 ** 127
    w[5] *= 2.0 ** -90  # blocks whose powers lie far apart
    p = (*gs.gs_rows_pack8(x), *(t.reshape(1, 96, -1) for t in gs.gs_rows_pack8(w)))
    offsets = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    _check_fwd(p, offsets, 200, None, torch.float32)
    _check_fwd(p, offsets, 200, None, torch.bfloat16)
    # and the other way about
    q = (*gs.gs_rows_pack8(w[:rows] if rows < 96 else w.repeat(8, 1)[:rows]),
         *(t.reshape(1, -1, t.shape[-1]) for t in gs.gs_rows_pack8(x[:5])))
    _check_fwd(q, offsets, 200, None, torch.float32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("rows", [5, 700])
def test_gradients_at_the_ends_of_bfloat16(rows, dtype):
    """Other gradients than float16's take the values as bfloat16 holds them:
    from 2^128 on (what float32's largest is kept as) its largest, below 2^-126
    in steps of 2^-133, which the lowest three bytes' values are finer than."""
    g = gen(51)
    i, o = 300, 96
    offsets = torch.tensor([0, 2, rows], dtype=torch.int32, device=DEV)
    x, w = randn(g, rows, i), randn(g, 2 * o, i)
    x[1, 3], x[2, 150], x[3, 290], w[5, 7] = 3.4e38, -3.4e38, 2.0 ** 127, -3.4e38
    low = (*gs.gs_rows_pack8(randn(g, rows, i) * 2.0 ** -121),
           *(t.reshape(2, o, -1) for t in gs.gs_rows_pack8(randn(g, 2 * o, i) * 2.0 ** -121)))
    for t in (low[1], low[3]):  # bytes 0 to 4
        t.view(torch.uint8).copy_(torch.randint(0, 5, t.shape, generator=g, device=DEV))
    high = (*gs.gs_rows_pack8(x), *(t.reshape(2, o, -1) for t in gs.gs_rows_pack8(w)))
    assert int(high[1].view(torch.uint8).max()) == 247
    for p, size in ((high, 2.0 ** -60), (low, 2.0 ** 110)):
        gys = (randn(g, rows, o) * size).to(dtype)
        exact = _values(p, i)
        held = _values(p, i, torch.bfloat16)
        assert not any(torch.equal(a, b) for a, b in zip(exact, held))
        refs, slacks = linear_bwd_ref(gys, held[0], offsets, held[1])
        grads = gs.gs_expert_linear8_bwd(gys, p[0], p[1], offsets, p[2], p[3], i)
        for got, ref, slack, what in zip(grads, refs, slacks, ("xs", "weight", "bias")):
            assert float(ref.abs().max()) > 1e-20
            check(got, ref, slack, what)


@pytest.mark.parametrize("rows", [5, 700])
def test_nan_stays_in_its_row(rows):
    offsets = torch.tensor([0, 2, rows], dtype=torch.int32, device=DEV)
    p = _packed(5, rows, 2, 300, 80, rows)
    clean = gs.gs_expert_linear8_fwd(p[0], p[1], offsets, p[2], p[3], 300)
    p[0].view(torch.uint8)[3, 140] = 0x7f
    ys = gs.gs_expert_linear8_fwd(p[0], p[1], offsets, p[2], p[3], 300)
    others = [r for r in range(rows) if r != 3]
    assert torch.equal(ys[others], clean[others]) and bool(torch.isnan(ys[3]).all())


@pytest.mark.parametrize("rows", [5, 700, 40000])
def test_what_lies_behind_the_last_channel_counts_for_nothing(rows):
    i, o = 259, 200  # rows of 272 bytes and four scales, three of them used
    offsets = torch.tensor([0, rows // 3, rows], dtype=torch.int32, device=DEV)
    p = _packed(18, rows, 2, i, o, rows)
    gys = randn(gen(18), rows, o, dtype=torch.bfloat16)
    run = lambda: (gs.gs_expert_linear8_fwd(p[0], p[1], offsets, p[2], p[3], i),
                   *gs.gs_expert_linear8_bwd(gys, p[0], p[1], offsets, p[2], p[3], i))
    clean = run()
    for q, s in ((p[0], p[1]), (p[2], p[3])):
        q.view(torch.uint8)[..., i:] = 0x7f
        s.view(torch.uint8)[..., 3:] = 255
    assert all(torch.equal(a, b) for a, b in zip(run(), clean))


@pytest.mark.parametrize("rows", [5, 700])
def test_a_scale_that_is_no_number(rows):
    """Byte 255: in a row, its answers; in a weight's, that column's."""
    offsets = torch.tensor([0, rows, rows], dtype=torch.int32, device=DEV)
    p = _packed(15, rows, 2, 300, 80, rows)
    clean = gs.gs_expert_linear8_fwd(p[0], p[1], offsets, p[2], p[3], 300)
    p[1].view(torch.uint8)[2, 1] = 255
    p[3].view(torch.uint8)[0, 7, 2] = 255
    p[3].view(torch.uint8)[1, 9, 0] = 255  # of an expert without rows
    ys = gs.gs_expert_linear8_fwd(p[0], p[1], offsets, p[2], p[3], 300)
    bad = torch.zeros_like(ys, dtype=torch.bool)
    bad[2] = True
    bad[:, 7] = True
    assert torch.equal(torch.isnan(ys), bad) and torch.equal(ys[~bad], clean[~bad])


def test_two_calls_at_once():
    """On two streams, without anything that they share."""
    _, offsets, _, _ = routed(16, 20000, 2, 8)
    p, q = _packed(16, 40000, 8, 256, 384, 40000), _packed(17, 40000, 8, 256, 384, 40000)
    gys = randn(gen(16), 40000, 384, dtype=torch.bfloat16)

    def run(r):
        return (gs.gs_expert_linear8_fwd(r[0], r[1], offsets, r[2], r[3], 256),
                *gs.gs_expert_linear8_bwd(gys, r[0], r[1], offsets, r[2], r[3], 256))

    want = run(p), run(q)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(3):
        for s, r in zip(streams, (p, q)):
            with torch.cuda.stream(s):
                got.append(run(r))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))


@pytest.mark.parametrize("rows", [16, 640])
def test_long_sums_of_one_sign(rows):
    """32768 positive terms, added up over at most 4096 of them, 32 at a time
    and each time cut off by less than 2^-23 of the sum (1.5e-5 in all), then
    once for each of those sums (8 roundings)."""
    g = gen(6)
    i, o = 32768, 64
    x, w = randn(g, rows, i).abs(), randn(g, o, i).abs()
    p = (*gs.gs_rows_pack8(x), *(t.reshape(1, o, -1) for t in gs.gs_rows_pack8(w)))
    offsets = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    ys = gs.gs_expert_linear8_fwd(p[0], p[1], offsets, p[2], p[3], i, dtype=torch.float32)
    xv, wv = _values(p, i)
    ref = xv @ wv[0].t()
    assert float(((ys - ref) / ref).abs().max()) <= 2e-5


def test_offsets_beyond_32_bits():
    rows, i, o = 2 ** 21 + 700, 1040, 1032  # 2.18e9 elements in and 2.16e9 out
    last = 150
    offsets = torch.tensor([0, 1000, rows - last, rows], dtype=torch.int32, device=DEV)
    g = gen(40)
    x = torch.zeros((rows, i), dtype=torch.bfloat16, device=DEV)
    x[:9], x[-last:] = randn(g, 9, i).bfloat16(), randn(g, last, i).bfloat16()
    xq, xs = gs.gs_rows_pack8(x)
    del x
    wq, ws = (t.reshape(3, o, -1) for t in gs.gs_rows_pack8(randn(g, 3 * o, i) / i ** 0.5))
    ys = gs.gs_expert_linear8_fwd(xq, xs, offsets, wq, ws, i)
    xv, wv = values_ref(xq[-last:], xs[-last:], i), values_ref(wq, ws, i)
    tail = torch.tensor([0, 0, 0, last], dtype=torch.int32, device=DEV)
    ref, slack = linear_ref(xv, tail, wv, None)
    check(ys[-last:], ref, slack, "ys")
    assert not bool(ys[9:1000].any()) and not bool(ys[2 ** 20:2 ** 20 + 1000].any())
    gys = ys.zero_()
    gys[-last:] = randn(g, last, o, dtype=torch.bfloat16)
    gx, gw, gb = gs.gs_expert_linear8_bwd(gys, xq, xs, offsets, wq, ws, i)
    refs, slacks = linear_bwd_ref(gys[-last:], xv, tail, wv)
    check(gx[-last:], refs[0], slacks[0], "grad_xs")
    check(gw, refs[1], slacks[1], "grad_weight")
    check(gb, refs[2], slacks[2], "grad_bias")
    assert not bool(gx[:1000].any()) and not bool(gx[2 ** 20:2 ** 20 + 1000].any())


def test_no_rows():
    p = _packed(7, 4, 3, 32, 40, 4)
    offsets = torch.zeros(4, dtype=torch.int32, device=DEV)
    none = p[0][:0], p[1][:0]
    assert gs.gs_expert_linear8_fwd(*none, offsets, p[2], p[3], 32).shape == (0, 40)
    gx, gw, gb = gs.gs_expert_linear8_bwd(torch.empty((0, 40), device=DEV), *none, offsets, p[2],
                                          p[3], 32)
    assert gx.shape == (0, 32) and not bool(gw.any()) and not bool(gb.any())


def test_offsets_that_lie_are_clamped():
    p = _packed(8, 50, 3, 64, 40, 50)
    lies = torch.tensor([-5, 70, 20, 4000], dtype=torch.int32, device=DEV)
    true = torch.tensor([0, 50, 50, 50], dtype=torch.int32, device=DEV)
    a = gs.gs_expert_linear8_fwd(p[0], p[1], lies, p[2], p[3], 64)
    assert torch.equal(a, gs.gs_expert_linear8_fwd(p[0], p[1], true, p[2], p[3], 64))


def test_outputs_of_any_alignment_repeat_and_streams():
    _, offsets, _, _ = routed(9, 900, 2, 4)
    p = _packed(9, 1800, 4, 192, 136, 1800)
    whole = gs.gs_expert_linear8_fwd(p[0], p[1], offsets, p[2], p[3], 192)
    room = torch.zeros(1800 * 136 + 1, dtype=torch.bfloat16, device=DEV)
    odd = room[1:].reshape(1800, 136)
    gs.gs_expert_linear8_fwd(p[0], p[1], offsets, p[2], p[3], 192, out=odd)
    assert torch.equal(odd, whole) and float(room[0]) == 0
    gys = randn(gen(9), 1800, 136, dtype=torch.bfloat16)
    shifted = torch.empty(1800 * 136 + 1, dtype=torch.bfloat16, device=DEV)[1:].reshape(1800, 136)
    shifted.copy_(gys)
    grads = gs.gs_expert_linear8_bwd(gys, p[0], p[1], offsets, p[2], p[3], 192)
    again = gs.gs_expert_linear8_bwd(shifted, p[0], p[1], offsets, p[2], p[3], 192)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = gs.gs_expert_linear8_fwd(p[0], p[1], offsets, p[2], p[3], 192, stream=side)
    grads2 = gs.gs_expert_linear8_bwd(gys, p[0], p[1], offsets, p[2], p[3], 192, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, whole) and all(torch.equal(a, b) for a, b in zip(grads, grads2))


def test_gradients_against_differences():
    """The product is linear in the values of xs and in bias, so differences
    along them have rounding errors only (float32 over 200 terms, 1e-4)."""
    _, offsets, _, _ = routed(10, 90, 2, 3)
    R, i, o = 180, 200, 50
    p = _packed(10, R, 3, i, o, R)
    q = _packed(11, R, 3, i, o, R)
    g = gen(12)
    gys = randn(g, R, o)
    gx, gw, gb = gs.gs_expert_linear8_bwd(gys, p[0], p[1], offsets, p[2], p[3], i)
    run = lambda a, w, b=None: gs.gs_expert_linear8_fwd(
        a[0], a[1], offsets, w[2], w[3], i, b, dtype=torch.float32).double()
    dot = lambda a, b: float((a.double() * b).sum())
    x0, x1 = values_ref(p[0], p[1], i), values_ref(q[0], q[1], i)
    w0, w1 = values_ref(p[2], p[3], i), values_ref(q[2], q[3], i)
    size = lambda a, b: 1e-4 * float(a.double().norm() * b.norm())
    diff = dot(gys, run(q, p) - run(p, p))
    assert abs(diff - dot(gx, x1 - x0)) <= size(gx, x1 - x0)
    diff = dot(gys, run(p, q) - run(p, p))
    assert abs(diff - dot(gw, w1 - w0)) <= size(gw, w1 - w0)
    b = randn(g, 3, o)
    diff = dot(gys, run(p, p, b) - run(p, p))
    assert abs(diff - dot(gb, b.double())) <= size(gb, b.double())


def test_captured_and_replayed():
    _, offsets, _, _ = routed(13, 1000, 2, 8)
    p = _packed(13, 2000, 8, 256, 320, 2000)
    gys = randn(gen(13), 2000, 320, dtype=torch.bfloat16)
    run = lambda: (gs.gs_expert_linear8_fwd(p[0], p[1], offsets, p[2], p[3], 256),
                   *gs.gs_expert_linear8_bwd(gys, p[0], p[1], offsets, p[2], p[3], 256))
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for seed in (1, 2):
        n = _packed(seed, 2000, 8, 256, 320, 2000)
        for a, b in zip(p, n):
            a.view(torch.uint8).copy_(b.view(torch.uint8))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, run()))


def test_a_layer_from_the_router_on():
    """The router's choice, rows packed and dispatched as they are, the
    products of both layers and the answer; 8-bit rows dispatch as 16-bit ones."""
    g = gen(30)
    T, D, H, O, E, k = 700, 96, 144, 24, 6, 2
    x, logits = randn(g, T, D), randn(g, T, E)
    keep = torch.rand(T, generator=g, device=DEV) > 0.2
    w1, w2 = randn(g, E * H, D) / D ** 0.5, randn(g, E * O, H) / H ** 0.5
    ids, weights, counts, _ = gs.gs_expert_route_fwd(logits, k, keep=keep)
    offsets, _, slots = gs.gs_expert_sort(ids, E)
    assert torch.equal(offsets[1:] - offsets[:-1], counts[:E])
    q, s = gs.gs_rows_pack8(x)
    xq = gs.gs_expert_dispatch(q.view(torch.float16), slots, offsets).view(q.dtype)
    xs = gs.gs_expert_dispatch(s.view(torch.float16), slots, offsets).view(s.dtype)
    p1 = [t.reshape(E, H, -1) for t in gs.gs_rows_pack8(w1)]
    p2 = [t.reshape(E, O, -1) for t in gs.gs_rows_pack8(w2)]
    h = gs.gs_expert_linear8_fwd(xq, xs, offsets, *p1, D, dtype=torch.float32).relu_()
    ys = gs.gs_expert_linear8_fwd(*gs.gs_rows_pack8(h), offsets, *p2, H, dtype=torch.float32)
    y = gs.gs_expert_combine(ys, slots, weights)
    # the same in 64 bits, the rounding of h to 8 bits taken over
    xv = values_ref(q, s, D)
    hv = values_ref(*gs.gs_rows_pack8(h), H)
    v1, v2 = values_ref(*p1, D), values_ref(*p2, H)
    want = torch.zeros((T, O), dtype=torch.float64, device=DEV)
    for t in range(T):
        for j in range(k):
            if int(ids[t, j]) < 0:
                continue
            e, r = int(ids[t, j]), int(slots[t, j])
            ref = torch.relu(v1[e] @ xv[t])
            assert float((h[r] - ref).abs().max()) <= 1e-5 * float(ref.abs().max())
            want[t] += weights[t, j].double() * (v2[e] @ hv[r])
    assert float((y - want).norm()) <= 1e-6 * float(want.norm())
    assert not bool(y[~keep].any())


def test_refusals():
    p = _packed(14, 20, 2, 64, 32, 20)
    offsets = torch.tensor([0, 10, 20], dtype=torch.int32, device=DEV)
    gys = torch.zeros((20, 32), device=DEV)
    fwd, bwd = gs.gs_expert_linear8_fwd, gs.gs_expert_linear8_bwd
    for bad in (lambda: fwd(p[0], p[1], offsets, p[2], p[3], 80),
                lambda: fwd(p[0], p[1], offsets[:2], p[2], p[3], 64),
                lambda: fwd(p[0], p[1][:10], offsets, p[2], p[3], 64),
                lambda: fwd(p[0].view(torch.uint8), p[1], offsets, p[2], p[3], 64),
                lambda: fwd(p[0], p[1], offsets, p[2][0], p[3], 64),
                lambda: fwd(p[0], p[1], offsets, p[2], p[3], 64, gys[:2]),
                lambda: fwd(p[0], p[1], offsets, p[2], p[3], 64, dtype=torch.float64),
                lambda: fwd(p[0], p[1], offsets, p[2], p[3], 64, out=gys),
                lambda: fwd(p[0].cpu(), p[1].cpu(), offsets, p[2], p[3], 64),
                lambda: bwd(gys[:19], p[0], p[1], offsets, p[2], p[3], 64),
                lambda: bwd(gys.double(), p[0], p[1], offsets, p[2], p[3], 64),
                lambda: bwd(gys, p[0], p[1], offsets, p[2], p[3], 63 + 17)):
        with pytest.raises(ValueError):
            bad()
