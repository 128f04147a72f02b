"""FP8 tensors with a scale for each block of 128, their products and the
experts' order, plain CPU definition (numpy, fp64).

TEST INFRASTRUCTURE ONLY: the tests may import this module; the library's
product path never does.  It shares no code with the CUDA path.

Elements are e4m3 (sign, 4 exponent bits of bias 7, 3 mantissa bits, no
infinity, magnitude code 127 NaN, largest 448).  With a the largest magnitude of
a block, at least 2^-100: scale = fp32(a / 448), code = v * fp32(448 / a)
rounded to nearest, ties to the even code.  A block with a NaN or an infinity
has a NaN scale and zero codes.
"""
import numpy as np

LARGEST, LEAST = 448.0, 2.0 ** -100


def grid():
    """The 127 magnitudes in code order."""
    c = np.arange(127)
    e, m = c >> 3, (c & 7) / 8
    return np.where(e == 0, m * 2.0 ** -6, (1 + m) * 2.0 ** (e - 7.0))


def _block(v):
    """One block (any shape, fp64) -> (codes uint8, scale float32)."""
    if not np.isfinite(v).all():
        return np.zeros(v.shape, np.uint8), np.float32(np.nan)
    a = np.float32(max(np.abs(v).max(), LEAST))
    q = np.abs(v) * np.float64(np.float32(LARGEST) / a)  # exact: 24 + 24 bits
    g = grid()
    hi = np.clip(np.searchsorted(g, q), 1, 126)
    mid = (g[hi - 1] + g[hi]) / 2
    code = np.where(q > mid, hi, np.where(q < mid, hi - 1, hi - (hi & 1)))
    return (code | np.signbit(v).astype(np.int64) << 7).astype(np.uint8), a / np.float32(LARGEST)


def quantize(v, block_rows=1):
    """v [N, K] (one expert's) -> (codes [N, K], scales [ceil(N / block_rows), ceil(K / 128)])."""
    v = np.asarray(v, np.float64)
    N, K = v.shape
    codes = np.empty((N, K), np.uint8)
    scales = np.empty((-(-N // block_rows), -(-K // 128)), np.float32)
    for r in range(scales.shape[0]):
        for b in range(scales.shape[1]):
            at = (slice(r * block_rows, (r + 1) * block_rows), slice(128 * b, 128 * b + 128))
            codes[at], scales[r, b] = _block(v[at])
    return codes, scales


def values(codes, scales, block_rows=1):
    """fp64 values of codes [N, K] with scales [ceil(N / block_rows), ceil(K / 128)]."""
    N, K = codes.shape
    g = np.append(grid(), np.nan)
    s = np.asarray(scales, np.float64)[np.arange(N)[:, None] // block_rows, np.arange(K)[None, :] // 128]
    return g[codes & 127] * np.where(codes >> 7, -1.0, 1.0) * s


def product(x, w, offsets=None):
    """(y, sum of magnitudes) of values x [M, K] and w [E, N, K]; rows outside
    every expert's are NaN."""
    ends = [0, x.shape[0]] if offsets is None else list(offsets)
    y = np.full((x.shape[0], w.shape[1]), np.nan)
    mag = y.copy()
    for e in range(w.shape[0]):
        a, b = ends[e], ends[e + 1]
        y[a:b] = x[a:b] @ w[e].T
        mag[a:b] = np.abs(x[a:b]) @ np.abs(w[e]).T
    return y, mag


def sort_experts(ids, E):
    """(offsets [E + 1], perm [A], pos [T, k]) of ids [T, k]."""
    flat = ids.reshape(-1)
    perm = [a for e in range(E) for a in range(flat.size) if flat[a] == e] if flat.size < 2000 else \
        [a for a in np.argsort(np.where((flat < 0) | (flat >= E), E, flat), kind="stable") if 0 <= flat[a] < E]
    pos = np.full(flat.size, -1, np.int32)
    pos[perm] = np.arange(len(perm))
    offsets = np.array([((flat >= 0) & (flat < e)).sum() for e in range(E + 1)], np.int32)
    return offsets, np.array(list(perm) + [-1] * (flat.size - len(perm)), np.int32), pos.reshape(ids.shape)


def combine(ys, pos, w, residual=None):
    """(out [T, H], sum of magnitudes) in fp64."""
    T, k = pos.shape
    out = np.zeros((T, ys.shape[1])) if residual is None else residual.astype(np.float64)
    mag = np.abs(out)
    for t in range(T):
        for j in range(k):
            if 0 <= pos[t, j] < T * k:
                out[t] += w[t, j] * ys[pos[t, j]]
                mag[t] += np.abs(w[t, j] * ys[pos[t, j]])
    return out, mag


def combine_backward(dout, ys, pos, w):
    """(dys with NaN in rows that no place names, dw, dw's sum of magnitudes)."""
    T, k = pos.shape
    dys, dw, mag = np.full(ys.shape, np.nan), np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            p = pos[t, j]
            if 0 <= p < T * k:
                dys[p] = w[t, j] * dout[t]
                dw[t, j] = dout[t] @ ys[p]
                mag[t, j] = np.abs(dout[t]) @ np.abs(ys[p])
    return dys, dw, mag


def swiglu(h):
    g, u = np.split(np.asarray(h, np.float64), 2, axis=1)
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * u
