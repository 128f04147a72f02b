"""Pins of oracle/fp8.py: hand-worked blocks, ties, the experts' order."""
import numpy as np
import pytest

from oracle import fp8


def test_grid():
    g = fp8.grid()
    assert len(g) == 127 and g[0] == 0 and g[1] == 2.0 ** -9 and g[8] == 2.0 ** -6 and g[126] == 448 and g[125] == 416
    assert (np.diff(g) > 0).all()


def test_block_by_hand():
    v = np.zeros((1, 130))
    v[0, :6] = [448, -224, 17, 19, 21, -0.0]
    v[0, 128:] = [-3.5, 1.75]
    c, s = fp8.quantize(v)
    assert s.dtype == np.float32 and s.shape == (1, 2) and s[0, 0] == 1 and s[0, 1] == np.float32(2.0 ** -7)
    # 17 and 19 are the middles of 16, 18, 20: to the even codes 16 and 20; 21 likewise to 20
    assert np.array_equal(fp8.values(c, s)[0, :6], [448, -224, 16, 20, 20, 0]) and c[0, 5] == 0x80
    assert np.array_equal(fp8.values(c, s)[0, 128:], [-3.5, 1.75])


def test_blocks_of_weights_and_extremes():
    v = np.zeros((130, 144))
    v[127, 127], v[128, 0], v[129, 143], v[0, 128] = 448, 896, np.inf, 2.0 ** -120
    c, s = fp8.quantize(v, 128)
    assert s.shape == (2, 2) and s[0, 0] == 1 and s[1, 0] == 2 and np.isnan(s[1, 1])
    assert s[0, 1] == np.float32(2.0 ** -100 / 448) and not c[0, 128:].any()
    assert c[127, 127] == 126 and c[128, 0] == 126 and not c[129, 143]
    assert np.isnan(fp8.values(c, s, 128)[128:, 128:]).all() and not np.isnan(fp8.values(c, s, 128)[:128]).any()


def test_error_is_at_most_half_a_step():
    v = np.random.default_rng(1).standard_normal((5, 300)) * 10
    c, s = fp8.quantize(v)
    step = np.repeat(s, 128, 1)[:, :300] * 2.0 ** -9
    assert (np.abs(fp8.values(c, s) - v) <= np.maximum(np.abs(v) * 2.0 ** -4 * (1 + 2.0 ** -20), step / 2)).all()


def test_sort_by_hand():
    ids = np.array([[2, 0], [-1, 2], [0, 5]], np.int32)
    o, perm, pos = fp8.sort_experts(ids, 3)
    assert list(o) == [0, 2, 2, 4] and list(perm) == [1, 4, 0, 3, -1, -1]
    assert pos.tolist() == [[2, 0], [-1, 3], [1, -1]]
    big = np.random.default_rng(2).integers(-1, 6, (700, 3)).astype(np.int32)
    small = [fp8.sort_experts(big[:600], 5), fp8.sort_experts(big, 5)]
    for (o, perm, pos), b in zip(small, (big[:600], big)):
        n = o[-1]
        assert np.array_equal(b.reshape(-1)[perm[:n]], np.repeat(np.arange(5), np.diff(o))) and (perm[n:] == -1).all()
        assert all((np.diff(perm[o[e]:o[e + 1]]) > 0).all() for e in range(5))
        assert np.array_equal(pos.reshape(-1)[perm[:n]], np.arange(n)) and (pos >= 0).sum() == n


def test_combine_and_its_gradient_by_differences():
    rng = np.random.default_rng(3)
    _, _, pos = fp8.sort_experts(np.array([[1, 0], [0, 1], [2, 1]], np.int32), 2)
    ys, w, dout = rng.standard_normal((6, 4)), rng.random((3, 2)), rng.standard_normal((3, 4))
    dys, dw, _ = fp8.combine_backward(dout, ys, pos, w)
    loss = lambda y, v: float((dout * fp8.combine(y, pos, v)[0]).sum())  # noqa: E731
    for t in (ys, w):
        grad = np.nan_to_num(dys) if t is ys else dw
        for i in np.ndindex(t.shape):
            up, down = t.copy(), t.copy()
            up[i] += 0.5
            down[i] -= 0.5
            d = (loss(up, w) - loss(down, w)) if t is ys else (loss(ys, up) - loss(ys, down))
            assert abs(d - grad[i]) < 1e-12
    assert np.isnan(dys[5]).all() and dw[2, 0] == 0 and pos[2, 0] == -1


@pytest.mark.parametrize("offsets", [None, [0, 2, 2, 5]])
def test_product(offsets):
    rng = np.random.default_rng(4)
    x, w = rng.standard_normal((6, 8)), rng.standard_normal((1 if offsets is None else 3, 4, 8))
    y, mag = fp8.product(x, w, offsets)
    expert = [0] * 6 if offsets is None else [0, 0, 2, 2, 2, None]
    for m in range(6):
        if expert[m] is None:
            assert np.isnan(y[m]).all()
        else:
            assert np.allclose(y[m], [sum(x[m, k] * w[expert[m], n, k] for k in range(8)) for n in range(4)])
            assert (mag[m] >= np.abs(y[m])).all()
