"""Microscaled (MX) formats, plain CPU definition (numpy, fp64).

TEST INFRASTRUCTURE ONLY: the tests may import this module; the library's
product path never does.  It shares no code with the CUDA path.

OCP Microscaling v1.0: blocks of 32 elements along a row share one scale
X = 2^(s - 127), s one byte (e8m0; 255 is NaN).  Elements are e4m3 (MXFP8:
sign, 4 exponent bits of bias 7, 3 mantissa bits, no infinity, magnitude code
127 NaN, largest 448) or e2m1 (MXFP4: sign, 2 exponent bits of bias 1, 1
mantissa bit, largest 6).  Quantisation takes s = floor(log2 max|v|) - emax
(emax 8 and 2), clamped to 2^-127, and rounds v / X to the nearest element,
ties to the even code, saturating.
"""
import numpy as np

MXFP8, MXFP4 = 0, 1
EMAX = {MXFP8: 8, MXFP4: 2}


def grid(fmt):
    """The format's magnitudes in code order (without NaN)."""
    if fmt == MXFP4:
        return np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    g = []
    for c in range(127):
        e, m = c >> 3, c & 7
        g.append(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(g)


def quantize(v, fmt):
    """v [R, K] fp64 -> (codes [R, K] one per element with the sign in the top
    bit, scale bytes [R, K/32])."""
    v = np.asarray(v, np.float64)
    R, K = v.shape
    b = v.reshape(R, K // 32, 32)
    bad = ~np.isfinite(b).all(-1)
    with np.errstate(invalid="ignore"):
        big = np.abs(np.where(bad[..., None], 0, b)).max(-1)
    _, e = np.frexp(big)  # big = m 2^e, m in [1/2, 1)
    s = np.where(big > 0, np.maximum(e - 1 - EMAX[fmt], -127), -127) + 127
    X = np.ldexp(1.0, s - 127)[..., None]
    a = np.abs(np.where(bad[..., None], 0, b)) / X
    g = grid(fmt)
    hi = np.clip(np.searchsorted(g, a), 1, len(g) - 1)   # g[hi - 1] < a <= g[hi], or the largest
    mid = (g[hi - 1] + g[hi]) / 2
    code = np.where(a > mid, hi, np.where(a < mid, hi - 1, np.where(hi % 2 == 0, hi, hi - 1)))
    sign = np.signbit(b).astype(np.int64) << (7 if fmt == MXFP8 else 3)
    code = np.where(bad[..., None], 0, code | sign)
    return code.reshape(R, K).astype(np.uint8), np.where(bad, 255, s).astype(np.uint8)


def values(codes, scales, fmt):
    """fp64 values of per-element codes [R, K] and row-major scales [R, K/32]."""
    R, K = codes.shape
    top = 7 if fmt == MXFP8 else 3
    g = np.append(grid(fmt), np.nan) if fmt == MXFP8 else grid(fmt)
    c = codes.astype(np.int64)
    X = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    v = g[c & ((1 << top) - 1)] * np.where(c >> top, -1.0, 1.0)
    return (v.reshape(R, K // 32, 32) * X[..., None]).reshape(R, K)


def pack(codes, fmt):
    """Per-element codes -> stored bytes: e2m1 two per byte, even k low."""
    return codes if fmt == MXFP8 else (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(stored, fmt):
    if fmt == MXFP8:
        return stored
    out = np.empty((stored.shape[0], 2 * stored.shape[1]), np.uint8)
    out[:, 0::2], out[:, 1::2] = stored & 15, stored >> 4
    return out


def tile_scales(s):
    """Row-major [R, nb] -> tiles of 128 rows x 4 blocks, padding zero."""
    R, nb = s.shape
    kt = -(-nb // 4)
    out = np.zeros(-(-R // 128) * kt * 512, np.uint8)
    for r in range(R):
        for b in range(nb):
            out[(r // 128 * kt + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4] = s[r, b]
    return out


def untile_scales(t, R, nb):
    kt = -(-nb // 4)
    r, b = np.arange(R)[:, None], np.arange(nb)[None, :]
    return t[(r // 128 * kt + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4]


def rmsnorm(x, residual, weight, eps):
    """(h, y) in fp64: h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight."""
    h = np.asarray(x, np.float64) + (0 if residual is None else np.asarray(residual, np.float64))
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    return h, y if weight is None else y * np.asarray(weight, np.float64)
