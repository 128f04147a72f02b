"""GPU parity of the microscaled operators (C ABI) against oracle/mx.py (fp64).

Quantisation and its reading back are exact, so they are compared bit for bit.
The norm's fp32 y carries a relative error of at most (H / 2 + 8) 2^-24 (each
addition of the sum of squares at most 2^-24, halved by the square root; around
it 1 / H, the mean and eps, halved too, the reciprocal root's two units, which
are 4 x 2^-24, and two products), so each element must lie between the
quantisations of y (1 -+ that).  A product of two elements is exact in fp32; a sum of K of them
in any order, each addition off by at most a whole step, is off by at most
K 2^-23 times the sum of magnitudes, and the result is rounded once (half a
step of the output's type)."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from int4_block_quantized_gb300 import binding as B
from oracle import mx

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = "cuda"
DT = [torch.float16, torch.bfloat16, torch.float32]
FMT = [B.MXFP8, B.MXFP4]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int4_block_quantized_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def f64(t):
    return t.detach().cpu().double().numpy()


def make(M, K, seed, dtype=torch.float32, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g) * torch.exp2(spread * torch.randn((M, 1), generator=g))
    return x.to(dtype)


def random_mx(M, K, fmt, seed, smin=112, smax=124):
    """(per-element codes, row-major scales) without NaN codes."""
    rng = np.random.default_rng(seed)
    c = rng.integers(0, 256 if fmt == B.MXFP8 else 16, (M, K)).astype(np.uint8)
    if fmt == B.MXFP8:
        c = np.where((c & 127) == 127, c ^ 1, c).astype(np.uint8)
    return c, rng.integers(smin, smax, (M, K // 32)).astype(np.uint8)


def to_dev(c, s, fmt):
    return (torch.from_numpy(np.ascontiguousarray(mx.pack(c, fmt))).to(DEV), torch.from_numpy(mx.tile_scales(s)).to(DEV))


def check_quantized(x64, codes, scales, fmt):
    rc, rs = mx.quantize(x64, fmt)
    assert np.array_equal(codes.cpu().numpy(), mx.pack(rc, fmt))
    assert np.array_equal(scales.cpu().numpy(), mx.tile_scales(rs))
    return rc, rs


# ------------------------------------------------------------ quantise, read
@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("M,K", [(1, 32), (1, 2048), (3, 96), (127, 160), (128, 128), (129, 1408), (300, 544)])
def test_quantize_and_dequant_exact(M, K, dtype, fmt):
    x = make(M, K, M * 7 + K, dtype)
    n = B.qmoe_mx_scale_bytes(M, K)
    codes, scales = B.qmoe_mx_quantize(x.to(DEV), fmt, scales=torch.full((n,), 77, dtype=torch.uint8, device=DEV))
    rc, rs = check_quantized(f64(x), codes, scales, fmt)
    ref = torch.from_numpy(mx.values(rc, rs, fmt))
    for out in DT:
        got = B.qmoe_mx_dequant(codes, scales, fmt, out).cpu()
        assert torch.equal(got, ref.to(torch.float32).to(out))  # exact in fp32, rounded once


@pytest.mark.parametrize("fmt", FMT)
def test_quantize_edges(fmt):
    """Ties, saturation, powers of two, zeros and signs, subnormals, the largest
    fp32, NaN and infinities: each in a block of its own."""
    g = mx.grid(fmt)
    mids = list((g[1:] + g[:-1]) / 2)
    rows = [list(g[-31:]) + [float(g[-1])], [0.0, -0.0], [2.0 ** -149, -2.0 ** -140], [2.0 ** -126],
            [float(np.finfo(np.float32).max), 1.0], [float(2.0 ** 100), 2.0 ** 90], [np.nan, 1.0], [np.inf, 1.0],
            [-np.inf, np.nan], [float(g[-1]) * 1.001], [float(g[-1]) * 1.1], [-1.0, 0.999999]]
    rows += [mids[i:i + 31] + [float(g[-1])] for i in range(0, len(mids), 31)]
    rows += [[-v for v in r] for r in rows]
    x = np.zeros((len(rows), 64), np.float32)
    for i, r in enumerate(rows):
        x[i, :len(r)] = r          # block 0
        x[i, 32:] = 1.5            # a neighbour that must not be touched by it
    codes, scales = B.qmoe_mx_quantize(torch.from_numpy(x).to(DEV), fmt)
    rc, rs = check_quantized(x.astype(np.float64), codes, scales, fmt)
    got = B.qmoe_mx_dequant(codes, scales, fmt, torch.float32).cpu().numpy()
    assert np.array_equal(got, mx.values(rc, rs, fmt).astype(np.float32), equal_nan=True)


@pytest.mark.parametrize("fmt", FMT)
def test_dequant_every_code_and_scale(fmt):
    n = 256 if fmt == B.MXFP8 else 16
    c = np.resize(np.arange(n, dtype=np.uint8), (256, 128))  # 256 codes in two rows: every code meets 128 scales
    s = np.arange(256, dtype=np.uint8)[:, None].repeat(4, 1)
    codes, scales = to_dev(c, s, fmt)
    got = B.qmoe_mx_dequant(codes, scales, fmt, torch.float32).cpu().numpy()
    with np.errstate(over="ignore"):
        ref = mx.values(c, s, fmt).astype(np.float32)
    assert np.array_equal(got, ref, equal_nan=True)


def test_quantize_beyond_32_bit_offsets():
    """More than 2^32 elements: the last rows as quantised alone."""
    K = 4128
    M = (1 << 32) // K + 300
    x = torch.zeros((M, K), dtype=torch.float16, device=DEV)
    tail = make(200, K, 5, torch.float16).to(DEV)
    x[-200:] = tail
    codes, scales = B.qmoe_mx_quantize(x, B.MXFP4)
    c1, s1 = B.qmoe_mx_quantize(tail, B.MXFP4)
    assert torch.equal(codes[-200:], c1) and not codes[:1000].any()
    a = B.qmoe_mx_untile_scales(scales, M, K)[-200:]
    assert torch.equal(a, B.qmoe_mx_untile_scales(s1, 200, K))
    v = B.qmoe_mx_dequant(codes, scales, B.MXFP4, torch.float16)
    assert torch.equal(v[-200:], B.qmoe_mx_dequant(c1, s1, B.MXFP4, torch.float16))


@pytest.mark.parametrize("R,K", [(1, 32), (128, 512), (131, 416), (1408, 2048)])
def test_scale_adapters(R, K):
    s = torch.randint(0, 256, (R, K // 32), generator=torch.Generator().manual_seed(R), dtype=torch.int32).to(torch.uint8)
    t = B.qmoe_mx_tile_scales(s.to(DEV))
    assert np.array_equal(t.cpu().numpy(), mx.tile_scales(s.numpy()))
    assert torch.equal(B.qmoe_mx_untile_scales(t, R, K).cpu(), s)


# ------------------------------------------------------------------- RMSNorm
def check_norm(x, residual, weight, eps, fmt, got):
    codes, scales, total = got
    T, H = x.shape
    h, y = mx.rmsnorm(f64(x), None if residual is None else f64(residual), None if weight is None else f64(weight), eps)
    if total is not None:
        # fp32 sum of two 16-bit numbers, rounded again: at most half a step and 2^-24 beyond
        bound = (torch.finfo(x.dtype).eps / 2 + 2.0 ** -24) * np.abs(h) + float(torch.finfo(x.dtype).smallest_normal) * 2.0 ** -10
        assert (np.abs(f64(total) - h) <= bound).all()
    r = (H / 2 + 8) * 2.0 ** -24
    v = np.abs(f64(B.qmoe_mx_dequant(codes, scales, fmt, torch.float32)))
    lc, ls = mx.quantize(y * (1 - r), fmt)
    hc, hs = mx.quantize(y * (1 + r), fmt)
    lo, hi = np.abs(mx.values(lc, ls, fmt)), np.abs(mx.values(hc, hs, fmt))
    ok = (v >= np.minimum(lo, hi)) & (v <= np.maximum(lo, hi))
    assert ok.all(), "%d elements outside" % int((~ok).sum())
    s = mx.untile_scales(scales.cpu().numpy(), T, H // 32)
    assert ((s == ls) | (s == hs)).all()
    assert int(scales.cpu().long().sum()) == int(s.astype(np.int64).sum())  # padding zero


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", DT[:2])
@pytest.mark.parametrize("T,H", [(1, 32), (1, 2048), (5, 96), (130, 1408), (17, 5632), (3, 8192), (2, 20000 // 32 * 32)])
def test_rmsnorm_mx(T, H, dtype, fmt):
    x, r = make(T, H, T + H, dtype, 1.0), make(T, H, T + H + 1, dtype, 1.0)
    w = (1 + 0.3 * torch.randn(H, generator=torch.Generator().manual_seed(H))).to(dtype)
    check_norm(x, r, w, 1e-6, fmt, B.qmoe_rmsnorm_mx(x.to(DEV), r.to(DEV), w.to(DEV), 1e-6, fmt))
    plain = B.qmoe_rmsnorm_mx(x.to(DEV), eps=1e-5, fmt=fmt)
    assert plain[2] is None
    check_norm(x, None, None, 1e-5, fmt, plain)


@pytest.mark.parametrize("T,H", [(3, 256), (2, 6144), (1, 40960)])
def test_rmsnorm_mx_in_place(T, H):
    """residual_out may be x or residual itself."""
    x, r = make(T, H, 1, torch.bfloat16).to(DEV), make(T, H, 2, torch.bfloat16).to(DEV)
    ref = B.qmoe_rmsnorm_mx(x, r)
    for which in (0, 1):
        a, b = x.clone(), r.clone()
        got = B.qmoe_rmsnorm_mx(a, b, residual_out=(a, b)[which])
        assert all(torch.equal(p, q) for p, q in zip(got, ref))
        assert torch.equal((a, b)[1 - which], (x, r)[1 - which])


def test_rmsnorm_mx_zero_and_non_finite_rows():
    x = make(4, 128, 3, torch.float16)
    x[1] = 0
    x[2, 5] = float("inf")
    x[3, 100] = float("nan")
    for fmt in FMT:
        codes, scales, _ = B.qmoe_rmsnorm_mx(x.to(DEV), eps=0.0 if fmt else 1e-6, fmt=fmt)
        v = B.qmoe_mx_dequant(codes, scales, fmt, torch.float32).cpu()
        assert torch.isfinite(v[0]).all()
        # 0 / sqrt(0 + eps): zeros, or NaN where eps is 0 too
        assert torch.isnan(v[1]).all() if fmt else not v[1].any()
        # inf / inf is NaN in its block, finite / inf is 0 elsewhere; a NaN spoils the row
        assert torch.isnan(v[2, :32]).all() and not v[2, 32:].any()
        assert torch.isnan(v[3]).all()


# ------------------------------------------------------------------- product
def check_product(xc, xs, xf, wc, ws, y, dtype):
    X, W = mx.values(xc, xs, xf), mx.values(wc, ws, B.MXFP4)
    ref = X @ W.T
    mag = np.abs(X) @ np.abs(W).T
    K = X.shape[1]
    bound = (1 + torch.finfo(dtype).eps) * K * 2.0 ** -23 * mag + torch.finfo(dtype).eps / 2 * np.abs(ref) + \
        float(torch.finfo(dtype).smallest_normal) * torch.finfo(dtype).eps / 2
    err = np.abs(f64(y) - ref)
    assert (err <= bound).all(), "worst %.3g of its bound" % float((err / bound).max())


def run_product(M, N, K, xf, dtype, seed=0, **kw):
    xc, xs = random_mx(M, K, xf, seed + 1)
    wc, ws = random_mx(N, K, B.MXFP4, seed + 2)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = B.qmoe_mx_matmul(*to_dev(xc, xs, xf), xf, *to_dev(wc, ws, B.MXFP4), dtype, status=st, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_product(xc, xs, xf, wc, ws, y, dtype)


@pytest.mark.parametrize("xf", FMT)
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (1, 8, 64), (1, 1408, 2048), (2, 129, 96), (3, 128, 128), (8, 200, 160),
                                   (9, 64, 288)])
def test_matmul_few_tokens(M, N, K, xf, dtype):
    run_product(M, N, K, xf, dtype, M + N + K)


@pytest.mark.parametrize("xf", FMT)
@pytest.mark.parametrize("M,N,K", [(16, 512, 1024), (17, 130, 416), (31, 384, 2048), (32, 256, 256), (33, 256, 5632),
                                   (64, 127, 512), (65, 129, 1408), (127, 255, 320), (128, 128, 640), (129, 257, 768),
                                   (200, 640, 2048), (333, 411, 1440), (512, 1408, 2048), (700, 300, 128), (1, 1, 128),
                                   (344, 62, 2912), (1019, 68, 4160), (400, 30, 4096), (2100, 130, 96)])
def test_matmul_tiles(M, N, K, xf):
    run_product(M, N, K, xf, (torch.float32, torch.bfloat16, torch.float16)[(M + N) % 3], M + N + K)


@pytest.mark.parametrize("xf", FMT)
@pytest.mark.parametrize("M,N,K", [(2600, 1900, 256), (2817, 1793, 128), (1281, 4001, 640), (5000, 1100, 416),
                                   (300, 9900, 32), (2561, 2050, 1152)])
def test_matmul_many_tiles(M, N, K, xf):
    """More tiles than SMs: several per CTA (or pair of CTAs), ragged last ones."""
    run_product(M, N, K, xf, (torch.float32, torch.bfloat16)[M % 2], M + N + K)


@pytest.mark.parametrize("xf", FMT)
@pytest.mark.parametrize("M,N,K", [(33, 40, 96), (70, 136, 160), (200, 1000, 256), (2600, 1912, 256), (2817, 1800, 128),
                                   (1281, 4008, 640), (129, 8, 128)])
@pytest.mark.parametrize("dtype", DT[:2])
def test_matmul_rows_of_y_on_16_bytes(M, N, K, xf, dtype):
    """N a multiple of 8 (y is then written in tiles), ragged tiles either way;
    and the same into a y that does not start on 16 bytes, which has to agree."""
    xc, xs = random_mx(M, K, xf, M + 1)
    wc, ws = random_mx(N, K, B.MXFP4, N + 2)
    x, w = to_dev(xc, xs, xf), to_dev(wc, ws, B.MXFP4)
    buf = torch.full((M * N + 64,), 7.0, dtype=dtype, device=DEV)
    y = B.qmoe_mx_matmul(*x, xf, *w, dtype, out=buf[16:16 + M * N].view(M, N))
    assert (buf[:16] == 7).all() and (buf[16 + M * N:] == 7).all()
    check_product(xc, xs, xf, wc, ws, y, dtype)
    other = torch.full((M * N + 64,), 7.0, dtype=dtype, device=DEV)
    assert torch.equal(B.qmoe_mx_matmul(*x, xf, *w, dtype, out=other[3:3 + M * N].view(M, N)), y)
    assert (other[:3] == 7).all() and (other[3 + M * N:] == 7).all()


@pytest.mark.parametrize("xf", FMT)
def test_matmul_scale_extremes(xf):
    """Scales across many binades between blocks, zero codes, the smallest scale."""
    M, N, K = 20, 150, 512
    xc, xs = random_mx(M, K, xf, 3, 60, 190)
    wc, ws = random_mx(N, K, B.MXFP4, 4, 100, 150)
    xc[4] = 0
    xs[5] = 0
    y = B.qmoe_mx_matmul(*to_dev(xc, xs, xf), xf, *to_dev(wc, ws, B.MXFP4), torch.float32)
    check_product(xc, xs, xf, wc, ws, y, torch.float32)
    assert not y[4].any()


@pytest.mark.parametrize("xf", FMT)
@pytest.mark.parametrize("M", [1, 20, 300])
def test_matmul_nan_scales_stay_in_their_rows(M, xf):
    N, K = 260, 288
    xc, xs = random_mx(M, K, xf, 5)
    wc, ws = random_mx(N, K, B.MXFP4, 6)
    ws[130, 8] = 255
    if M > 1:
        xs[M // 2, 0] = 255
    y = f64(B.qmoe_mx_matmul(*to_dev(xc, xs, xf), xf, *to_dev(wc, ws, B.MXFP4), torch.float32))
    assert np.isnan(y[:, 130]).all()
    bad = np.zeros_like(y, bool)
    bad[:, 130] = True
    if M > 1:
        bad[M // 2] = True
    assert np.array_equal(np.isnan(y), bad)


@pytest.mark.parametrize("M,N,K,xf", [(3, 70, 256, 0), (140, 200, 160, 1), (300, 333, 512, 0)])
def test_matmul_writes_y_alone(M, N, K, xf):
    """The elements around y stay as they were; y is any element-aligned place;
    what lies behind the scales' last row and block does not matter."""
    xc, xs = random_mx(M, K, xf, 7)
    wc, ws = random_mx(N, K, B.MXFP4, 8)
    x, w = to_dev(xc, xs, xf), to_dev(wc, ws, B.MXFP4)
    ref = B.qmoe_mx_matmul(*x, xf, *w, torch.float16)
    buf = torch.full((M * N + 200,), 7.0, dtype=torch.float16, device=DEV)
    out = buf[99:99 + M * N].view(M, N)
    B.qmoe_mx_matmul(*x, xf, *w, torch.float16, out=out)
    assert torch.equal(out, ref) and (buf[:99] == 7).all() and (buf[99 + M * N:] == 7).all()
    # padding rows of the scale tiles: any bytes, NaN among them
    dirty = x[1].clone().view(-1, 32, 4, 4)
    r = torch.arange(128, device=DEV).view(4, 32).t().reshape(1, 32, 4, 1) + \
        128 * (torch.arange(dirty.shape[0], device=DEV) // -(-K // 128)).view(-1, 1, 1, 1)
    dirty = torch.where(r >= M, torch.full_like(dirty, 255), dirty).reshape(-1).contiguous()
    assert torch.equal(B.qmoe_mx_matmul(x[0], dirty, xf, *w, torch.float16), ref)


@pytest.mark.parametrize("M,N,K,xf", [(1, 1408, 2048, 0), (300, 500, 1024, 1)])
def test_matmul_is_reproducible_on_streams_and_in_graphs(M, N, K, xf):
    xc, xs = random_mx(M, K, xf, 9)
    wc, ws = random_mx(N, K, B.MXFP4, 10)
    x, w = to_dev(xc, xs, xf), to_dev(wc, ws, B.MXFP4)
    ref = B.qmoe_mx_matmul(*x, xf, *w)
    side = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(6):  # two streams at once, sharing inputs
        side[i % 2].wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side[i % 2]):
            outs.append(B.qmoe_mx_matmul(*x, xf, *w))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    g = torch.cuda.CUDAGraph()
    out = torch.zeros_like(ref)
    with torch.cuda.graph(g):
        B.qmoe_mx_matmul(*x, xf, *w, out=out)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


def at_16(t):
    """A copy of t that starts on a 16-byte boundary and on no 32-byte one."""
    n = 16 // t.element_size()
    buf = torch.empty(t.numel() + 2 * n, dtype=t.dtype, device=DEV)
    return buf[n:n + t.numel()].view(t.shape).copy_(t)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", DT)
def test_streams_on_16_byte_boundaries(dtype, fmt):
    """Every pointer off a 32-byte boundary gives what aligned ones give."""
    M, K = 37, 416
    x, r = make(M, K, 1, dtype).to(DEV), make(M, K, 2, dtype).to(DEV)
    ref = B.qmoe_mx_quantize(x, fmt)
    out = tuple(at_16(t) for t in ref)
    got = B.qmoe_mx_quantize(at_16(x), fmt, codes=out[0].zero_(), scales=out[1].zero_())
    assert got[0].data_ptr() % 32 == 16 and all(torch.equal(a, b) for a, b in zip(got, ref))
    v = B.qmoe_mx_dequant(*ref, fmt, dtype)
    assert torch.equal(B.qmoe_mx_dequant(*got, fmt, dtype, out=at_16(torch.zeros_like(v))), v)
    if dtype != torch.float32:
        w = make(1, K, 3, dtype).to(DEV)[0]
        ref = B.qmoe_rmsnorm_mx(x, r, w, fmt=fmt)
        got = B.qmoe_rmsnorm_mx(at_16(x), at_16(r), at_16(w), fmt=fmt, residual_out=at_16(x), codes=at_16(ref[0]).zero_(),
                                scales=at_16(ref[1]).zero_())
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("xf", FMT)
@pytest.mark.parametrize("M,N,K", [(5, 300, 512), (150, 700, 1024), (2700, 1900, 256)])
def test_matmul_on_16_byte_boundaries(M, N, K, xf):
    """Weights off a 32-byte boundary take the other way in; sums are in another
    order only where the split of K differs, so fp32 results agree to rounding."""
    x, w = to_dev(*random_mx(M, K, xf, 4), xf), to_dev(*random_mx(N, K, B.MXFP4, 5), B.MXFP4)
    xc, xs = random_mx(M, K, xf, 4)
    wc, ws = random_mx(N, K, B.MXFP4, 5)
    y = B.qmoe_mx_matmul(at_16(x[0]), at_16(x[1]), xf, at_16(w[0]), at_16(w[1]), torch.float32)
    check_product(xc, xs, xf, wc, ws, y, torch.float32)


@pytest.mark.parametrize("M", [2, 70])
def test_matmul_nan_code_spoils_its_row(M):
    """e4m3 has a NaN code; the product's row is NaN, the others are not."""
    N, K = 140, 256
    xc, xs = random_mx(M, K, B.MXFP8, 6)
    xc[M - 1, 77] = 0xff
    y = f64(B.qmoe_mx_matmul(*to_dev(xc, xs, B.MXFP8), B.MXFP8, *to_dev(*random_mx(N, K, B.MXFP4, 7), B.MXFP4), torch.float32))
    assert np.isnan(y[M - 1]).all() and np.isfinite(y[:M - 1]).all()


def test_first_calls_of_a_process_inside_a_capture():
    """Nothing of the operators needs a call before the capture."""
    code = """
import sys; sys.path.insert(0, %r)
import torch
from int4_block_quantized_gb300 import binding as B
g = torch.Generator(device="cuda").manual_seed(1)
x, r, w = (torch.randn(s, generator=g, device="cuda").half() for s in ((5, 512), (5, 512), (300, 512)))
graph = torch.cuda.CUDAGraph()
def run():
    c, s, total = B.qmoe_rmsnorm_mx(x, r)
    wc, ws = B.qmoe_mx_quantize(w, B.MXFP4)
    return total, B.qmoe_mx_matmul(c, s, B.MXFP8, wc, ws), B.qmoe_mx_dequant(wc, ws, B.MXFP4), B.qmoe_mx_untile_scales(ws, 300, 512)
with torch.cuda.graph(graph):
    out = run()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, run()))
""" % ROOT
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300)


def test_graphs_on_two_streams_at_once():
    """Two captured graphs share weights and run side by side."""
    M, N, K = 40, 1408, 2048
    w = to_dev(*random_mx(N, K, B.MXFP4, 2), B.MXFP4)
    xs = [to_dev(*random_mx(M, K, B.MXFP8, 3 + i), B.MXFP8) for i in range(2)]
    ref = [B.qmoe_mx_matmul(*x, B.MXFP8, *w) for x in xs]
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(B.qmoe_mx_matmul(*x, B.MXFP8, *w))
        graphs.append(g)
    side = [torch.cuda.Stream() for _ in range(2)]
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for g, s in zip(graphs, side):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, ref))


def test_product_beside_the_layer_on_another_stream():
    """The layer's tensor-core kernels (router, grouped GEMM) and the product each
    take tensor memory; on two streams at once both finish with their own results."""
    from int4_block_quantized_gb300 import synthetic as S
    wl = S.WORKLOADS["prefill"]
    layer = dict(S.make_layer(wl, seed=1, device=DEV))
    ws = B.Workspace(wl.T, wl.H, wl.I, wl.E, wl.k, device=DEV)
    _, w_ref, ids_ref = B.qmoe_forward(layer, ws=ws, return_routing=True)
    # pairs of CTAs; clusters along K
    cases = [(2600, 1912, 512), (40, 1408, 2048)]
    args = [(to_dev(*random_mx(m, k, B.MXFP8, 1), B.MXFP8), to_dev(*random_mx(n, k, B.MXFP4, 2), B.MXFP4)) for m, n, k in cases]
    refs = [B.qmoe_mx_matmul(*x, B.MXFP8, *w) for x, w in args]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got, routed = [], []
    for i in range(30):
        routed.append(B.qmoe_forward(layer, ws=ws, return_routing=True)[1:])
        with torch.cuda.stream(side):
            x, w = args[i % 2]
            got.append(B.qmoe_mx_matmul(*x, B.MXFP8, *w))
    torch.cuda.synchronize()
    assert ws.status() == (0, 0)
    assert all(torch.equal(w, w_ref) and torch.equal(i, ids_ref) for w, i in routed)
    assert all(torch.equal(y, refs[i % 2]) for i, y in enumerate(got))


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("T", [1, 5, 160])
@pytest.mark.parametrize("fmt", FMT)
def test_norm_feeds_product_and_layer(T, fmt):
    """One block as it would run: the norm adds the layer's output to the
    residual, its microscaled output goes through an MXFP4 projection and back,
    eager and captured; checked against the oracle on the codes that were
    handed on."""
    H, N = 512, 384
    x, r = make(T, H, 11, torch.bfloat16, 1.0).to(DEV), make(T, H, 12, torch.bfloat16, 1.0).to(DEV)
    w1 = B.qmoe_mx_quantize((0.05 * make(N, H, 13, torch.float32, 0.0)).to(DEV), B.MXFP4)
    w2 = B.qmoe_mx_quantize((0.05 * make(H, N, 14, torch.float32, 0.0)).to(DEV), B.MXFP4)

    def block():
        c, s, total = B.qmoe_rmsnorm_mx(x, r, fmt=fmt)
        y = B.qmoe_mx_matmul(c, s, fmt, *w1, torch.bfloat16)
        c2, s2 = B.qmoe_mx_quantize(y, fmt)
        z = B.qmoe_mx_matmul(c2, s2, fmt, *w2, torch.bfloat16)
        c3, s3, total = B.qmoe_rmsnorm_mx(z, total, fmt=fmt, residual_out=total)
        return c, s, y, c2, s2, z, c3, s3, total

    eager = block()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = block()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, captured))
    c, s, y, c2, s2, z, c3, s3, total = eager

    def host(codes, scales, f):
        codes = mx.unpack(codes.cpu().numpy(), f)
        return codes, mx.untile_scales(scales.cpu().numpy(), codes.shape[0], codes.shape[1] // 32)
    check_product(*host(c, s, fmt), fmt, *host(*w1, B.MXFP4), y, torch.bfloat16)
    check_quantized(f64(y), c2, s2, fmt)
    check_product(*host(c2, s2, fmt), fmt, *host(*w2, B.MXFP4), z, torch.bfloat16)
    first = B.qmoe_rmsnorm_mx(x, r, fmt=fmt)[2]
    check_norm(z.cpu(), first.cpu(), None, 1e-6, fmt, (c3, s3, total))


def test_refusals_on_the_device():
    x = make(4, 64, 1, torch.float16).to(DEV)
    c, s = B.qmoe_mx_quantize(x)
    w = B.qmoe_mx_quantize(x, B.MXFP4)
    bad = [lambda: B.qmoe_mx_quantize(x.t()), lambda: B.qmoe_mx_quantize(x[:, :48].contiguous()),
           lambda: B.qmoe_mx_quantize(x.double()), lambda: B.qmoe_mx_quantize(x, 3), lambda: B.qmoe_mx_quantize(x[0]),
           lambda: B.qmoe_mx_quantize(x[:, ::2]), lambda: B.qmoe_mx_quantize(x[:0]),
           lambda: B.qmoe_mx_dequant(c, s[:-1], B.MXFP8), lambda: B.qmoe_mx_dequant(c, s, B.MXFP8, torch.float64),
           lambda: B.qmoe_mx_dequant(c, s.cpu(), B.MXFP8), lambda: B.qmoe_rmsnorm_mx(x, x[:2]),
           lambda: B.qmoe_rmsnorm_mx(x, x.bfloat16()), lambda: B.qmoe_rmsnorm_mx(x, weight=x[0, :32]),
           lambda: B.qmoe_rmsnorm_mx(x.float()), lambda: B.qmoe_rmsnorm_mx(x, eps=-1.0),
           lambda: B.qmoe_mx_matmul(c, s, B.MXFP4, *w), lambda: B.qmoe_mx_matmul(c, s, B.MXFP8, w[0][:, :16].contiguous(), w[1]),
           lambda: B.qmoe_mx_matmul(c, s, B.MXFP8, *w, torch.float64),
           lambda: B.qmoe_mx_matmul(c, s, B.MXFP8, *w, out=torch.empty(4, 4, device=DEV)),
           lambda: B.qmoe_mx_quantize(torch.zeros(65 * 64, dtype=torch.float16, device=DEV)[4:4 + 256].view(4, 64))]
    for i, call in enumerate(bad):
        with pytest.raises(B.QMoEError) as e:
            call()
        assert e.value.code == 1, i
