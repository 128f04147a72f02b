"""Pins of the MX oracle (oracle/mx.py), CPU only: the element tables against
the format definitions, hand-worked blocks, ties, saturation, the scale rule at
powers of two and at the clamp, non-finite blocks, and the layouts."""
import numpy as np
import pytest
import torch

from oracle import mx


def test_element_tables():
    e4m3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(mx.grid(mx.MXFP8), e4m3) and mx.grid(mx.MXFP8)[-1] == 448
    assert list(mx.grid(mx.MXFP4)) == [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def _block(first, rest=0.0):
    return np.array([first + [rest] * (32 - len(first))], np.float64)


def test_hand_block_mxfp4():
    # largest 6 -> floor(log2) = 2, emax 2, X = 1; ties 0.25 -> 0, 0.75 -> 1,
    # 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4 (even codes)
    c, s = mx.quantize(_block([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.3, -6, 0.74]), mx.MXFP4)
    assert s[0, 0] == 127
    assert list(c[0, :11]) == [7, 0, 2, 2, 4, 4, 6, 6, 8 | 1, 8 | 7, 1]
    assert bytes(mx.pack(c, mx.MXFP4)[0, :4]) == bytes([0x07, 0x22, 0x44, 0x66])
    # 7.9 saturates at 6: floor(log2 7.9) = 2
    c, s = mx.quantize(_block([7.9, 8 - 2 ** -20]), mx.MXFP4)
    assert s[0, 0] == 127 and list(c[0, :2]) == [7, 7]
    # 8 is the next power of two: X = 2, code of 4
    c, s = mx.quantize(_block([8.0]), mx.MXFP4)
    assert s[0, 0] == 128 and c[0, 0] == 6


def test_hand_block_mxfp8():
    c, s = mx.quantize(_block([256, 449, 511.9, -448, 17, 2 ** -9, 2 ** -10, 3 * 2 ** -10]), mx.MXFP8)
    assert s[0, 0] == 127
    v = mx.values(c, s, mx.MXFP8)[0]
    assert list(v[:8]) == [256, 448, 448, -448, 16, 2 ** -9, 0, 2 ** -8]


def test_scale_clamp_and_zero():
    for fmt in (mx.MXFP8, mx.MXFP4):
        c, s = mx.quantize(_block([0.0, -0.0]), fmt)
        assert s[0, 0] == 0 and c[0, 0] == 0 and c[0, 1] == (128 if fmt == mx.MXFP8 else 8)
        c, s = mx.quantize(_block([2.0 ** -126, 2.0 ** -149]), fmt)
        assert s[0, 0] == 0 and mx.values(c, s, fmt)[0, 0] == 2.0 ** -126
        assert mx.quantize(_block([2.0 ** 127]), fmt)[1][0, 0] == 254 - mx.EMAX[fmt]


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_non_finite_block_reads_nan(bad):
    v = np.ones((2, 64))
    v[0, 40] = bad
    for fmt in (mx.MXFP8, mx.MXFP4):
        c, s = mx.quantize(v, fmt)
        assert s[0, 1] == 255 and not c[0, 32:].any() and s[0, 0] != 255 and (s[1] != 255).all()
        w = mx.values(c, s, fmt)
        assert np.isnan(w[0, 32:]).all() and (w[0, :32] == 1).all()


def test_values_of_all_codes():
    c = np.arange(256, dtype=np.uint8).reshape(8, 32)
    v = mx.values(c, np.full((8, 1), 127, np.uint8), mx.MXFP8).reshape(-1)
    ref = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, ref, equal_nan=True)


def test_quantised_values_are_nearest():
    rng = np.random.default_rng(0)
    v = rng.standard_normal((16, 256)) * np.exp2(rng.integers(-20, 20, (16, 1)))
    for fmt in (mx.MXFP8, mx.MXFP4):
        c, s = mx.quantize(v, fmt)
        g = mx.grid(fmt)
        X = np.ldexp(1.0, s.astype(int) - 127).repeat(32, 1)
        near = np.abs(np.abs(v / X)[..., None] - g).min(-1)
        assert np.array_equal(np.abs(np.abs(v) - np.abs(mx.values(c, s, fmt))) / X, near)


def test_layouts():
    rng = np.random.default_rng(1)
    for R, nb in ((1, 1), (130, 5), (256, 8)):
        s = rng.integers(1, 255, (R, nb), dtype=np.uint8)
        t = mx.tile_scales(s)
        assert t.size == -(-R // 128) * -(-nb // 4) * 512
        assert np.array_equal(mx.untile_scales(t, R, nb), s)
        assert int(t.astype(int).sum()) == int(s.astype(int).sum())  # padding is zero
    s = np.zeros((128, 4), np.uint8)
    s[33, 2] = 9
    assert mx.tile_scales(s)[1 * 16 + 1 * 4 + 2] == 9
    c = rng.integers(0, 16, (3, 64), dtype=np.uint8)
    assert np.array_equal(mx.unpack(mx.pack(c, mx.MXFP4), mx.MXFP4), c)


def test_rmsnorm_definition():
    h, y = mx.rmsnorm([[3.0, 4.0]], [[0.0, 0.0]], [2.0, 1.0], 0.0)
    r = np.sqrt(12.5)
    assert np.allclose(y, [[6 / r, 4 / r]], rtol=1e-15) and np.array_equal(h, [[3.0, 4.0]])
