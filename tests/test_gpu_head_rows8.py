"""Rows kept in 8 bits (gs_rows_pack8 / gs_rows_unpack8) against their 64-bit
form: bit for bit, there is one right answer."""

import pytest
import torch

from head8_util import cut, pack_ref, values_ref
from head_util import DEV, TYPES, gen, randn, sliced
from tile_gaussian_splat_gb300 import binding as gs

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (1, 64), (5, 3), (7, 16), (129, 64), (64, 131), (33, 256), (40, 515), (300, 32),
          (1000, 1024), (9, 1023), (17, 2050), (3, 16384), (4099, 24), (2500, 128), (31, 1500),
          (2, 65536), (77, 48), (513, 129)]


def _same(a, b):
    return bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


def _check(x):
    rows, ch = x.shape
    q, scales = gs.gs_rows_pack8(x)
    wide, blocks = (ch + 15) // 16 * 16, (ch + 127) // 128
    assert q.shape == (rows, wide) and scales.shape == (rows, (ch + 511) // 512 * 4)
    values, byte = pack_ref(x)
    assert torch.equal(scales.view(torch.uint8)[:, :blocks].long(), byte)
    assert not bool(scales.view(torch.uint8)[:, blocks:].any())
    assert not bool(q.view(torch.uint8)[:, ch:].any())
    assert _same(values_ref(q, scales, ch), values)
    for dtype in TYPES:
        y = gs.gs_rows_unpack8(q, scales, ch, dtype)
        assert y.dtype == dtype and _same(y, cut(values, dtype).to(dtype))
    return q, scales


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows,ch", SHAPES)
def test_there_and_back(rows, ch, dtype):
    for pad in (0, 3, 8):
        g = gen(100 * rows + ch + pad)
        x = randn(g, rows, ch) * torch.exp(4 * randn(g, rows, 1))
        x[torch.rand((rows, 1), generator=g, device=DEV).expand(rows, ch) < 0.1] = 0
        q, scales = _check(sliced(x.to(dtype), pad))
        wide = torch.full((rows, ch + pad), 3.0, dtype=dtype, device=DEV)
        gs.gs_rows_unpack8(q, scales, ch, dtype, out=wide[:, pad:])
        assert _same(wide[:, pad:], gs.gs_rows_unpack8(q, scales, ch, dtype))
        assert bool((wide[:, :pad] == 3).all())


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_the_range_of_the_type(dtype):
    info = torch.finfo(dtype)
    tiny = info.smallest_normal * 2.0 ** -(8 if dtype == torch.float32 else 4)
    x = torch.zeros((12, 140), dtype=dtype, device=DEV)
    x[0, :] = info.max
    x[1, 5], x[1, 6] = info.max, -info.max
    x[2, :] = tiny
    x[3, 0], x[3, 1] = tiny, info.max
    x[4, 130] = info.smallest_normal
    # where a block's power changes: 448, 449 or 450 (the type's next), 447
    x[5, 0], x[6, 0], x[7, 0] = 448.0, 450.0, 446.0
    # halfway between two e4m3 values, normal and below
    x[8, 0] = 448.0
    x[8, 1:9] = torch.tensor([17.0, 19.0, 1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10, -17.0,
                              -2.0 ** -10]).to(dtype)
    x[9] = torch.arange(140, device=DEV) - 70
    x[10] = -0.0
    _check(x)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("ch", [64, 131, 300])
def test_what_is_not_finite_stays_where_it_is(ch, dtype):
    g = gen(ch)
    x = randn(g, 30, ch, dtype=dtype)
    clean = gs.gs_rows_unpack8(*gs.gs_rows_pack8(x), ch, dtype)
    x[3, 5], x[4, 0], x[5, ch - 1] = float("nan"), float("inf"), -float("inf")
    x[6] = float("nan")
    x[7] = float("inf")
    _check(x)
    y = gs.gs_rows_unpack8(*gs.gs_rows_pack8(x), ch, dtype)
    assert torch.equal(torch.isnan(y), ~torch.isfinite(x))
    others = [r for r in range(30) if r not in (3, 4, 5, 6, 7)]
    assert torch.equal(y[others], clean[others])


def test_every_code_and_scale():
    q = torch.arange(256, dtype=torch.int32).to(torch.uint8).to(DEV).reshape(1, 256).repeat(256, 1)
    byte = torch.arange(256, dtype=torch.int32).to(torch.uint8).to(DEV)[:, None].repeat(1, 4)
    q8, s8 = q.view(torch.float8_e4m3fn), byte.view(torch.float8_e8m0fnu)
    values = values_ref(q8[:255], s8[:255], 256)
    for dtype in TYPES:
        y = gs.gs_rows_unpack8(q8, s8, 256, dtype)
        assert _same(y[:255], cut(values, dtype).to(dtype))
        assert bool(torch.isnan(y[255]).all())  # a scale that is no number


def test_no_rows_images_and_other_streams():
    empty = torch.empty((0, 33), device=DEV)
    q, scales = gs.gs_rows_pack8(empty)
    assert q.shape == (0, 48) and scales.shape == (0, 4)
    assert gs.gs_rows_unpack8(q, scales, 33).shape == (0, 33)
    g = gen(3)
    image = randn(g, 2, 37, 53, 67)
    q, scales = gs.gs_rows_pack8(image[..., 3:])
    assert q.shape == (2, 37, 53, 64) and scales.shape == (2, 37, 53, 4)
    y = gs.gs_rows_unpack8(q, scales, 64, torch.float32)
    values, _ = pack_ref(image[..., 3:].reshape(-1, 64))
    assert torch.equal(y.reshape(-1, 64).double(), values)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q2, s2 = gs.gs_rows_pack8(image[..., 3:], stream=side)
    y2 = gs.gs_rows_unpack8(q2, s2, 64, torch.float32, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(y, y2)
    assert torch.equal(scales.view(torch.uint8), s2.view(torch.uint8))


def test_offsets_beyond_32_bits():
    rows, ch = 2 ** 21 + 5, 1040
    x = torch.zeros((rows, ch), dtype=torch.bfloat16, device=DEV)  # 2.18e9 elements
    x[-3:] = randn(gen(4), 3, ch, dtype=torch.bfloat16)
    q, scales = gs.gs_rows_pack8(x)
    y = gs.gs_rows_unpack8(q, scales, ch, torch.bfloat16)
    values, _ = pack_ref(x[-3:])
    assert torch.equal(y[-3:].double(), values)
    assert not bool(q[:-3].view(torch.uint8).any()) and not bool(y[:-3].any())


def test_refusals():
    x = torch.zeros((4, 40), device=DEV)
    q, scales = gs.gs_rows_pack8(x)
    for bad in (lambda: gs.gs_rows_pack8(x.double()), lambda: gs.gs_rows_pack8(x.t()),
                lambda: gs.gs_rows_pack8(x.cpu()), lambda: gs.gs_rows_unpack8(q, scales, 50),
                lambda: gs.gs_rows_unpack8(q, scales[:3], 40),
                lambda: gs.gs_rows_unpack8(q.view(torch.uint8), scales, 40),
                lambda: gs.gs_rows_unpack8(q, scales.view(torch.uint8), 40),
                lambda: gs.gs_rows_unpack8(q, scales, 40, torch.float64),
                lambda: gs.gs_rows_unpack8(q.cpu(), scales.cpu(), 40),
                lambda: gs.gs_rows_unpack8(q, scales, 40, out=x[:, :39])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(gs.GsError, match="INVALID_ARG"):
        gs.gs_rows_pack8(torch.zeros((1, 65537), device=DEV))
    raw = torch.zeros(4 * 48 + 8, dtype=torch.uint8, device=DEV)
    with pytest.raises(gs.GsError, match="INVALID_ARG"):  # off a 16-byte boundary
        gs.gs_rows_unpack8(raw[8:].view(torch.float8_e4m3fn).reshape(4, 48), scales, 40)
