"""GPU parity of the FP8 experts' operators (C ABI) against oracle/fp8.py (fp64).

Quantisation of given values and reading back are exact, so they are compared bit
for bit.  SwiGLU in fp32 carries a relative error of at most 9 2^-24 (the
exponential's 2 units, which are 4 2^-24, the reciprocal's unit, 2 2^-24, and a
rounding each of the sum and the two products), so a value's code must be the
nearest to a quotient within that and 2^-22 (the scale's, of the same error and a
rounding, is on one side of it) of it.  A product: each addition within a block of 128 off
by at most a whole step (2^-23), then the product of the scales, its product with
the block's sum and the sum over blocks, each half a step: with nb blocks at most
(128 + nb + 4) 2^-23 times the sum of magnitudes; the result is rounded once
(half a step of the output's type).  A combined row: k + 1 products and sums, each
half a step; a weight's gradient: H products and sums."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from int4_block_quantized_gb300 import binding as B
from oracle import fp8

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = "cuda"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
DT = [F16, BF16, F32]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int4_block_quantized_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def f64(t):
    return t.detach().cpu().double().numpy()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def make(M, K, seed, dtype=F32, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((M, K), generator=g) * torch.exp2(spread * torch.randn((M, 1), generator=g))).to(dtype)


def same_scales(got, want):
    return np.array_equal(got.cpu().numpy(), want, equal_nan=True)


def ids_of(T, k, E, seed, drop=0.0):
    rng = np.random.default_rng(seed)
    w = rng.random(E) ** 3 + 1e-3  # some experts busy, some nearly idle
    ids = rng.choice(E, (T, k), p=w / w.sum()).astype(np.int32)
    ids[rng.random((T, k)) < drop] = -1
    return ids


# ------------------------------------------------------------ quantise, read
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("M,K", [(1, 16), (1, 2048), (3, 144), (5, 112), (127, 128), (33, 1408), (300, 272), (2, 8192)])
def test_quantize_and_dequant_exact(M, K, dtype):
    x = make(M, K, M * 7 + K, dtype)
    codes, scales = B.qmoe_fp8_quantize(x.to(DEV))
    rc, rs = fp8.quantize(f64(x))
    assert np.array_equal(codes.cpu().numpy(), rc) and same_scales(scales, rs)
    ref = torch.from_numpy(fp8.values(rc, rs))  # 4 + 24 bits: exact in fp64, rounded once by the reader's product
    for out in DT:
        assert torch.equal(B.qmoe_fp8_dequant(codes, scales, out).cpu(), ref.float().to(out))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("E,N,K", [(1, 1, 16), (1, 128, 128), (2, 129, 144), (3, 200, 400), (1, 300, 2048), (2, 127, 112)])
def test_quantize_weights_exact(E, N, K, dtype):
    w = make(E * N, K, E + N + K, dtype, 1.0)
    codes, scales = B.qmoe_fp8_quantize_weights(w.view(E, N, K).to(DEV))
    vals = B.qmoe_fp8_dequant(codes, scales, F32).cpu()
    for e in range(E):
        rc, rs = fp8.quantize(f64(w[e * N:(e + 1) * N]), 128)
        assert np.array_equal(codes[e].cpu().numpy(), rc) and same_scales(scales[e], rs)
        assert torch.equal(vals[e], torch.from_numpy(fp8.values(rc, rs, 128)).float())
    flat = B.qmoe_fp8_quantize_weights(w[:N].to(DEV).contiguous())
    assert torch.equal(flat[0], codes[0]) and torch.equal(flat[1], scales[0])


def test_quantize_edges():
    """Ties, saturation, zeros and signs, subnormals, tiny and huge blocks, NaN and
    infinities: each in a block of its own beside one that it must not touch."""
    g = fp8.grid()
    mids = list((g[1:] + g[:-1]) / 2)
    rows = [list(g[-100:]) + [448.0], [0.0, -0.0], [2.0 ** -149, -2.0 ** -140], [2.0 ** -126], [2.0 ** -100, 2.0 ** -101],
            [2.0 ** -99, -2.0 ** -109, 2.0 ** -117], [float(np.finfo(np.float32).max), 1.0, 2.0 ** 118], [2.0 ** 100, 2.0 ** 91, 1.0],
            [np.nan, 1.0], [np.inf, 1.0], [-np.inf, np.nan], [-1.0, 0.999999, 1e-3], [3.0, 1.0, 0.1]]
    rows += [mids[i:i + 100] + [448.0] for i in range(0, len(mids), 100)]
    rows += [[-v for v in r] for r in rows]
    x = np.zeros((len(rows), 272), np.float32)
    for i, r in enumerate(rows):
        x[i, :len(r)] = r
        x[i, 128:256] = 1.5
        x[i, 256:] = r[0]
    rc, rs = fp8.quantize(x.astype(np.float64))
    codes, scales = B.qmoe_fp8_quantize(dev(x))
    assert np.array_equal(codes.cpu().numpy(), rc) and same_scales(scales, rs)
    assert np.array_equal(f64(B.qmoe_fp8_dequant(codes, scales, F32)).astype(np.float32), fp8.values(rc, rs).astype(np.float32), equal_nan=True)
    rc, rs = fp8.quantize(x.astype(np.float64), 128)
    codes, scales = B.qmoe_fp8_quantize_weights(dev(x))
    assert np.array_equal(codes.cpu().numpy(), rc) and same_scales(scales, rs)


@pytest.mark.parametrize("dtype", DT)
def test_quantize_values_next_to_a_border(dtype):
    """Values whose fp32 product with the reciprocal falls on a border between two
    codes while the exact one does not: bf16 quotients hit borders often."""
    g = torch.Generator().manual_seed(5)
    x = (torch.randint(1, 256, (4096, 128), generator=g) * torch.exp2(torch.randint(-4, 5, (4096, 128), generator=g).float())).to(dtype)
    rc, rs = fp8.quantize(f64(x))
    codes, scales = B.qmoe_fp8_quantize(x.to(DEV))
    assert np.array_equal(codes.cpu().numpy(), rc) and same_scales(scales, rs)


def test_dequant_every_code():
    c = np.resize(np.arange(256, dtype=np.uint8), (260, 256))
    s = np.exp2(np.random.default_rng(1).integers(-130, 100, (260, 2))).astype(np.float32)
    s[3, 1] = np.nan
    with np.errstate(over="ignore"):
        ref = fp8.values(c, s).astype(np.float32)
    got = B.qmoe_fp8_dequant(dev(c), dev(s), F32).cpu().numpy()
    assert np.array_equal(got, ref, equal_nan=True)


@pytest.mark.parametrize("T,k,K", [(1, 4, 2048), (5, 1, 16), (70, 3, 144), (300, 8, 256)])
def test_quantize_to_places(T, k, K):
    """A token's codes and scales at each of its places; other rows stay."""
    x = make(T, K, T + k, BF16).to(DEV)
    ids = ids_of(T, k, 7, T, 0.2)
    _, perm, pos = B.qmoe_sort_experts(dev(ids), 7)
    codes = torch.full((T * k, K), 99, dtype=torch.uint8, device=DEV)
    scales = torch.full((T * k, -(-K // 128)), 7.0, device=DEV)
    B.qmoe_fp8_quantize(x, pos, codes=codes, scales=scales)
    c, s = B.qmoe_fp8_quantize(x)
    n = int((perm >= 0).sum())
    token = (perm[:n] // k).long()
    assert torch.equal(codes[:n], c[token]) and torch.equal(scales[:n], s[token])
    assert (codes[n:] == 99).all() and (scales[n:] == 7).all()


def test_places_outside_are_ignored():
    T, k, K = 6, 2, 64
    x = make(T, K, 1, F16).to(DEV)
    pos = torch.tensor([[0, 12], [-1, 3], [2 ** 31 - 1, 5], [-2 ** 31, 7], [9, 11], [13, 1]], dtype=torch.int32, device=DEV)
    buf = torch.full((3, T * k, K), 99, dtype=torch.uint8, device=DEV)
    sc = torch.full((3, T * k, 1), 7.0, device=DEV)
    B.qmoe_fp8_quantize(x, pos, codes=buf[1], scales=sc[1])
    xs = torch.full((3, T * k, K), 7.0, dtype=F16, device=DEV)
    B.qmoe_dispatch(x, pos, out=xs[1])
    named = {0: 0, 3: 1, 5: 2, 7: 3, 9: 4, 11: 4, 1: 5}
    c, s = B.qmoe_fp8_quantize(x)
    for r in range(T * k):
        if r in named:
            assert torch.equal(buf[1, r], c[named[r]]) and torch.equal(sc[1, r], s[named[r]]) and torch.equal(xs[1, r], x[named[r]])
        else:
            assert (buf[1, r] == 99).all() and (sc[1, r] == 7).all() and (xs[1, r] == 7).all()
    assert (buf[::2] == 99).all() and (sc[::2] == 7).all() and (xs[::2] == 7).all()
    ys = make(T * k, K, 2, F32).to(DEV)
    out = B.qmoe_combine(ys, pos)
    ref = fp8.combine(f64(ys), pos.cpu().numpy(), np.ones((T, k)))
    assert (np.abs(f64(out) - ref[0]) <= 3 * 2.0 ** -24 * ref[1]).all()
    dys, dw = B.qmoe_combine_backward(x, ys, pos, dys=torch.full_like(ys, 7.0))
    for r in range(T * k):
        assert torch.equal(dys[r], x[named[r]].float()) if r in named else (dys[r] == 7).all()
    assert dw[0, 1] == 0 and dw[1, 0] == 0 and dw[2, 0] == 0 and dw[3, 0] == 0 and dw[5, 0] == 0


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("M,I", [(1, 16), (1, 1408), (37, 144), (200, 768), (3, 5632)])
def test_swiglu(M, I, dtype):
    h = make(M, 2 * I, M + I, dtype, 1.0)
    h[0, :I] *= 30  # deep in both tails
    y = fp8.swiglu(f64(h))
    codes, scales = B.qmoe_fp8_quantize_swiglu(h.to(DEV))
    s, c = f64(scales), codes.cpu().numpy()
    r = 9 * 2.0 ** -24
    a = np.stack([np.abs(y[:, 128 * b:128 * b + 128]).max(1) for b in range(s.shape[1])], 1)
    assert (np.abs(s - np.maximum(a, 2.0 ** -100) / 448) <= (r + 2.0 ** -24) * s).all()
    g, mag = fp8.grid(), c & 127
    mids = np.concatenate([[0], (g[1:] + g[:-1]) / 2, [np.inf]])
    q = np.abs(y) / np.repeat(s, 128, 1)[:, :I]
    slack = (1 + r) * (1 + r + 2.0 ** -22)
    assert (mids[mag] <= q * slack).all() and (q / slack <= mids[mag + 1]).all()
    assert ((c >> 7 == 1) == (y < 0))[np.abs(q) > 2.0 ** -9].all()


def test_swiglu_extremes():
    """gate far below zero (the product with up must not overflow first), far above,
    NaN and infinities in one half."""
    h = np.zeros((6, 256), np.float32)
    h[:, :128], h[:, 128:] = 1.0, 1.0
    h[0, 0], h[0, 128] = -3e38, 3e38
    h[1, 0], h[1, 128] = 1e20, 1e17
    h[2, 5], h[3, 133], h[4, 5] = np.nan, np.inf, -200.0
    h[5] = 0
    codes, scales = B.qmoe_fp8_quantize_swiglu(dev(h))
    v = f64(B.qmoe_fp8_dequant(codes, scales, F32))
    y = fp8.swiglu(h)
    assert v[0, 0] == 0 and abs(v[0, 1] - y[0, 1]) < 2.0 ** -4 and abs(v[1, 0] / 1e37 - 1) < 1e-6
    assert np.isnan(v[2]).all() and np.isnan(v[3]).all() and v[4, 5] == 0 and not v[5].any()


# ------------------------------------------------------------------- product
def random_fp8(shape, seed, smin=-8, smax=-3):
    """Codes without NaN (uniform) and scales over some binades, not powers of two."""
    rng = np.random.default_rng(seed)
    c = rng.integers(0, 256, shape).astype(np.uint8)
    return np.where((c & 127) == 127, c ^ 1, c).astype(np.uint8), \
        lambda *s: (rng.uniform(1, 2, s) * np.exp2(rng.integers(smin, smax, s))).astype(np.float32)


def operands(M, N, K, E=1, seed=0, grouped=False):
    xc, xs = random_fp8((M, K), seed + 1)
    wc, ws = random_fp8((E, N, K), seed + 2)
    nb = -(-K // 128)
    return xc, xs(M, nb), wc, ws(E, -(-N // 128), nb)


def bound_of(ref, mag, K, dtype):
    i = torch.finfo(dtype)
    nb = -(-K // 128)
    return (1 + i.eps) * (128 + nb + 4) * 2.0 ** -23 * mag + i.eps / 2 * np.abs(ref) + float(i.smallest_normal) * i.eps / 2


def check_product(ops, y, dtype, offsets=None):
    xc, xs, wc, ws = ops
    X = fp8.values(xc, xs)
    W = np.stack([fp8.values(c, s, 128) for c, s in zip(wc, ws)])
    ref, mag = fp8.product(X, W, offsets)
    live = ~np.isnan(mag[:, 0])
    err, b = np.abs(f64(y) - ref)[live], bound_of(ref, mag, xc.shape[1], dtype)[live]
    assert (err <= b).all(), "worst %.3g of its bound, %d outside" % (float((err / b).max()), int((err > b).sum()))


def run_dense(M, N, K, dtype, seed=0):
    ops = operands(M, N, K, 1, seed)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    buf = torch.full((M * N + 64,), 7.0, dtype=dtype, device=DEV)
    y = B.qmoe_fp8_matmul(dev(ops[0]), dev(ops[1]), dev(ops[2][0]), dev(ops[3][0]), dtype, out=buf[32:32 + M * N].view(M, N), status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and (buf[:32] == 7).all() and (buf[32 + M * N:] == 7).all()
    check_product(ops, y, dtype)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 8, 64), (1, 1408, 2048), (2, 129, 96), (3, 128, 128), (8, 200, 272), (9, 64, 400),
                                   (16, 130, 144)])
def test_matmul_few_tokens(M, N, K, dtype):
    run_dense(M, N, K, dtype, M + N + K)


@pytest.mark.parametrize("M,N,K", [(17, 130, 416), (31, 384, 2048), (32, 256, 256), (33, 256, 5632), (64, 127, 512), (65, 129, 1408),
                                   (127, 255, 336), (128, 128, 640), (129, 257, 768), (200, 640, 2048), (333, 411, 1424),
                                   (512, 1408, 2048), (700, 300, 128), (257, 1, 128), (344, 62, 2912), (1019, 68, 4160),
                                   (400, 30, 4096), (2100, 130, 96), (300, 9900, 32), (128, 4104, 1024), (70, 136, 8208)])
def test_matmul_tiles(M, N, K):
    run_dense(M, N, K, DT[(M + N) % 3], M + N + K)


@pytest.mark.parametrize("M,N,K", [(2600, 1904, 256), (2817, 1793, 128), (1281, 4001, 640), (5000, 1104, 416), (2561, 2050, 1152),
                                   (4096, 2048, 384)])
def test_matmul_many_tiles(M, N, K):
    """More tiles than SMs: several per CTA (or pair of CTAs), ragged last ones."""
    run_dense(M, N, K, (F32, BF16)[M % 2], M + N + K)


def test_matmul_any_place_of_y():
    """y on any element, also off 16 bytes, gives the same bits."""
    for M, N, K in ((40, 264, 256), (300, 1032, 384), (3, 136, 512)):
        ops = [dev(a[0] if a.ndim == 3 else a) for a in operands(M, N, K)]
        ref = B.qmoe_fp8_matmul(*ops, F16)
        for at in (1, 3, 8):
            buf = torch.full((M * N + 64,), 7.0, dtype=F16, device=DEV)
            assert torch.equal(B.qmoe_fp8_matmul(*ops, F16, out=buf[at:at + M * N].view(M, N)), ref)
            assert (buf[:at] == 7).all() and (buf[at + M * N:] == 7).all()


def at_offset(t, n):
    """A copy of t that starts n bytes behind a 256-byte boundary."""
    n //= t.element_size()
    buf = torch.empty(t.numel() + n, dtype=t.dtype, device=DEV)
    return buf[n:].view(t.shape).copy_(t)


@pytest.mark.parametrize("M,N,K", [(5, 300, 512), (150, 700, 1024), (2700, 1900, 384), (9, 128, 1296)])
def test_matmul_on_the_least_alignment(M, N, K):
    """Codes on 16-byte boundaries and scales on 4-byte ones."""
    ops = [dev(a[0] if a.ndim == 3 else a) for a in operands(M, N, K)]
    ref = B.qmoe_fp8_matmul(*ops, F32)
    got = B.qmoe_fp8_matmul(at_offset(ops[0], 16), at_offset(ops[1], 4), at_offset(ops[2], 48), at_offset(ops[3], 12), F32)
    assert torch.equal(got, ref)


GROUPED = [(1, 4, 60, 256, 512), (3, 2, 8, 130, 272), (16, 4, 60, 192, 256), (100, 4, 8, 264, 400), (64, 8, 256, 64, 128),
           (512, 4, 60, 320, 256), (300, 1, 3, 1000, 144), (1000, 2, 4, 129, 640), (2, 1, 256, 128, 2048), (257, 8, 5, 72, 1024)]


@pytest.mark.parametrize("T,k,E,N,K", GROUPED)
def test_matmul_grouped(T, k, E, N, K):
    dtype = DT[(T + N) % 3]
    ids = ids_of(T, k, E, T + E, 0.15 if T > 2 else 0)
    offsets, perm, _ = fp8.sort_experts(ids, E)
    M = T * k
    ops = operands(M, N, K, E, T)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full((M, N), 7.0, dtype=dtype, device=DEV)
    y = B.qmoe_fp8_matmul(*(dev(a) for a in ops), dtype, offsets=dev(offsets), out=out, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_product(ops, y, dtype, offsets)
    assert (y[offsets[-1]:] == 7).all()  # rows behind the last expert's stay


@pytest.mark.parametrize("counts,M", [([0, 0, 0], 5), ([0, 9, 0], 9), ([5, 0, 0], 5), ([0, 0, 300], 300), ([1, 1, 1], 3), ([128, 1, 127], 300),
                                      ([257, 0, 64], 400), ([33, 31, 32], 96)])
def test_matmul_grouped_counts(counts, M):
    """Experts without rows, with all of them, tiles that end with an expert."""
    N, K, E = 200, 272, len(counts)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    ops = operands(M, N, K, E, M)
    out = torch.full((M, N), 7.0, dtype=BF16, device=DEV)
    y = B.qmoe_fp8_matmul(*(dev(a) for a in ops), BF16, offsets=dev(offsets), out=out)
    check_product(ops, y, BF16, offsets)
    assert (y[offsets[-1]:] == 7).all() and B.qmoe_fp8_status() == (0, 0)


def test_matmul_rows_before_the_first_expert_stay():
    M, N, K = 50, 72, 128
    offsets = np.array([7, 20, 41], np.int32)
    ops = operands(M, N, K, 2, 3)
    y = B.qmoe_fp8_matmul(*(dev(a) for a in ops), F32, offsets=dev(offsets), out=torch.full((M, N), 7.0, device=DEV))
    check_product(ops, y, F32, offsets)
    assert (y[:7] == 7).all() and (y[41:] == 7).all()


@pytest.mark.parametrize("offsets", [[0, 5, 11], [-3, 5, 10], [0, 7, 2], [0, 2 ** 31 - 1, 10], [-2 ** 31, 2 ** 31 - 1, -2 ** 31]])
def test_matmul_bad_offsets_are_reported(offsets):
    M, N, K = 10, 72, 128
    ops = [dev(a) for a in operands(M, N, K, 2, 3)]
    buf = torch.full((3, M, N), 7.0, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    B.qmoe_fp8_matmul(*ops, F32, offsets=off, out=buf[1], status=st)
    assert int(st.item()) == 2 and (buf == 7).all()
    B.qmoe_fp8_matmul(*ops, F32, offsets=off, out=buf[1])
    assert B.qmoe_fp8_status() == (6, 2) and B.qmoe_fp8_status() == (0, 0)
    good = torch.tensor([0, 5, 10], dtype=torch.int32, device=DEV)
    assert torch.isfinite(B.qmoe_fp8_matmul(*ops, F32, offsets=good, status=st.zero_())).all() and int(st.item()) == 0


@pytest.mark.parametrize("M", [1, 20, 300])
def test_matmul_nan_stays_where_it_enters(M):
    N, K = 260, 400
    xc, xs, wc, ws = operands(M, N, K, 1, 5)
    ws[0, 1, 3] = np.nan          # outputs 128 .. 255
    wc[0, 5, 9] = 0x7f            # output 5
    bad = np.zeros((M, N), bool)
    bad[:, 128:256] = bad[:, 5] = True
    if M > 1:
        xs[M // 2, 0], xc[M - 1, 399] = np.nan, 0xff
        bad[M // 2] = bad[M - 1] = True
    y = f64(B.qmoe_fp8_matmul(dev(xc), dev(xs), dev(wc[0]), dev(ws[0]), F32))
    assert np.array_equal(np.isnan(y), bad)


def test_matmul_nan_in_other_experts_rows():
    """Tiles reach over an expert's last row into the next one's; nothing of these
    rows, nor of rows behind the last expert's, enters."""
    counts, N, K = [3, 20, 130], 136, 272
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    M = int(offsets[-1]) + 40
    ops = operands(M, N, K, 3, 9)
    ref = B.qmoe_fp8_matmul(*(dev(a) for a in ops), BF16, offsets=dev(offsets), out=torch.zeros((M, N), dtype=BF16, device=DEV))
    for e in range(4):  # rows of expert e (3: behind the last) spoiled
        a, b = offsets[e], offsets[e + 1] if e < 3 else M
        xc, xs = ops[0].copy(), ops[1].copy()
        xc[a:b], xs[a:b] = 0x7f, np.nan
        wc = ops[2].copy()
        if e < 3:
            wc[e] = 0xff
        y = B.qmoe_fp8_matmul(dev(xc), dev(xs), dev(wc), dev(ops[3]), BF16, offsets=dev(offsets), out=torch.zeros((M, N), dtype=BF16, device=DEV))
        assert torch.equal(y[:a], ref[:a]) and torch.equal(y[b:], ref[b:])
        assert e == 3 or torch.isnan(y[a:b]).all()


def test_matmul_scale_extremes():
    """Scales over many binades between blocks, zero codes, zero scales."""
    M, N, K = 20, 150, 512
    xc, xs = random_fp8((M, K), 3, -60, 40)
    wc, ws = random_fp8((1, N, K), 4, -30, 20)
    xs, ws = xs(M, 4), ws(1, 2, 4)
    xc[4], xs[5] = 0, 0
    y = B.qmoe_fp8_matmul(dev(xc), dev(xs), dev(wc[0]), dev(ws[0]), F32)
    check_product((xc, xs, wc, ws), y, F32)
    assert not y[4:6].any()


@pytest.mark.parametrize("M,N,K,E", [(1, 1408, 2048, 1), (300, 500, 1024, 1), (2100, 2048, 512, 1), (64, 256, 512, 8)])
def test_matmul_is_reproducible_on_streams_and_in_graphs(M, N, K, E):
    ops = [dev(a) for a in operands(M, N, K, E, 9)]
    off = None
    if E > 1:
        off = dev(np.linspace(0, M - 3, E + 1).astype(np.int32))
    else:
        ops = [a[0] if a.dim() == 3 else a for a in ops]
    zeros = lambda: torch.zeros((M, N), dtype=BF16, device=DEV)  # noqa: E731
    ref = B.qmoe_fp8_matmul(*ops, offsets=off, out=zeros())
    side = [torch.cuda.Stream() for _ in range(2)]
    outs = [zeros() for _ in range(6)]
    for i in range(6):  # two streams at once, sharing inputs
        side[i % 2].wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side[i % 2]):
            B.qmoe_fp8_matmul(*ops, offsets=off, out=outs[i])
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    graphs, res = [], [zeros(), zeros()]
    for out in res:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            B.qmoe_fp8_matmul(*ops, offsets=off, out=out)
        graphs.append(g)
    for _ in range(2):  # two captured graphs side by side
        for i in range(2):
            res[i].zero_()
            side[i].wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(r, ref) for r in res)


def test_matmul_offsets_change_between_replays():
    """A captured grouped product reads its offsets at each replay."""
    M, N, K, E = 200, 192, 256, 6
    ops = operands(M, N, K, E, 4)
    d = [dev(a) for a in ops]
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    out = torch.zeros((M, N), device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.qmoe_fp8_matmul(*d, F32, offsets=off, out=out)
    for seed in range(4):
        o = np.sort(np.random.default_rng(seed).integers(0, M + 1, E + 1)).astype(np.int32)
        off.copy_(torch.from_numpy(o))
        g.replay()
        check_product(ops, out, F32, o)


# ------------------------------------------------------------ sort, dispatch
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 4, 60), (7, 2, 3), (33, 8, 256), (512, 4, 60), (1024, 4, 60), (1025, 4, 60), (5000, 3, 128),
                                   (16384, 8, 256), (40000, 1, 2)])
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_sort_experts(T, k, E, drop):
    ids = ids_of(T, k, E, T + E, drop)
    got = B.qmoe_sort_experts(dev(ids), E)
    for a, b in zip(got, fp8.sort_experts(ids, E)):
        assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("ids", [np.full((50, 2), -1), np.full((50, 2), 3), np.full((3000, 2), 59), np.full((3000, 2), 60),
                                 np.array([[-2 ** 31, 2 ** 31 - 1], [60, 59], [0, 0]])])
def test_sort_experts_one_sided(ids):
    """No assignment at all, one expert for all, the same expert twice in a row."""
    ids = ids.astype(np.int32)
    for a, b in zip(B.qmoe_sort_experts(dev(ids), 60), fp8.sort_experts(ids, 60)):
        assert np.array_equal(a.cpu().numpy(), b)


def test_sort_experts_agrees_with_the_router():
    T, H, E, k = 300, 256, 60, 4
    g = torch.Generator(device=DEV).manual_seed(1)
    x, rw = torch.randn((T, H), generator=g, device=DEV).half(), (0.1 * torch.randn((H, E), generator=g, device=DEV)).half()
    _, ids, off, perm = B.qmoe_route(x, rw, k)
    o, p, pos = B.qmoe_sort_experts(ids, E)
    assert torch.equal(o, off) and torch.equal(p, perm)
    assert torch.equal(pos.view(-1)[perm.long()], torch.arange(T * k, device=DEV, dtype=torch.int32))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,k,E,H", [(1, 4, 60, 2048), (3, 1, 2, 8), (40, 3, 5, 24), (200, 8, 60, 1000), (513, 4, 60, 256)])
def test_dispatch_and_combine(T, k, E, H, dtype):
    rng = np.random.default_rng(T)
    ids = ids_of(T, k, E, T, 0.2 if T > 3 else 0)
    _, perm, pos = B.qmoe_sort_experts(dev(ids), E)
    n = int((perm >= 0).sum())
    x = make(T, H, 1, dtype, 1.0).to(DEV)
    xs = B.qmoe_dispatch(x, pos, out=torch.full((T * k, H), 7.0, dtype=dtype, device=DEV))
    assert torch.equal(xs[:n], x[(perm[:n] // k).long()]) and (xs[n:] == 7).all()
    p, w = pos.cpu().numpy(), rng.random((T, k)).astype(np.float32)
    ys = make(T * k, H, 2, dtype, 1.0)
    ys[n:] = float("nan")  # rows that go nowhere are not read
    eps = torch.finfo
    for res_dt in DT:
        res = make(T, H, 3, res_dt, 1.0)
        for r, weights in ((res, w), (None, w), (res, None)):
            out = B.qmoe_combine(ys.to(DEV), pos, None if weights is None else dev(weights), None if r is None else r.to(DEV))
            assert out.dtype is (dtype if r is None else res_dt)
            ref, mag = fp8.combine(f64(ys), p, np.ones((T, k)) if weights is None else weights.astype(np.float64), None if r is None else f64(r))
            i = eps(out.dtype)
            b = (1 + i.eps) * (k + 1) * 2.0 ** -24 * mag + i.eps / 2 * np.abs(ref) + float(i.smallest_normal) * i.eps / 2
            assert (np.abs(f64(out) - ref) <= b).all()
        inplace = res.to(DEV)
        full = B.qmoe_combine(ys.to(DEV), pos, dev(w), inplace.clone())
        assert torch.equal(B.qmoe_combine(ys.to(DEV), pos, dev(w), inplace, out=inplace), full)
        dout = make(T, H, 4, res_dt, 1.0)
        ysd = torch.where(torch.isnan(ys), torch.zeros_like(ys), ys).to(DEV)
        ysd[n:] = float("nan")
        dys, dw = B.qmoe_combine_backward(dout.to(DEV), ysd, pos, dev(w), dys=torch.full((T * k, H), 7.0, dtype=dtype, device=DEV),
                                          dw=torch.full((T, k), 7.0, device=DEV))
        rys, rw, mag = fp8.combine_backward(f64(dout), f64(ys), p, w.astype(np.float64))
        i = eps(dtype)
        b = (i.eps / 2 + 2.0 ** -23) * np.abs(rys) + float(i.smallest_normal) * i.eps / 2
        assert (np.abs(f64(dys) - rys)[:n] <= b[:n]).all() and (dys[n:] == 7).all()
        assert (np.abs(f64(dw) - rw) <= H * 2.0 ** -24 * mag).all() and not dw[pos < 0].any()
    dx = B.qmoe_dispatch_backward(ys.to(DEV), pos)
    assert torch.equal(dx, B.qmoe_combine(ys.to(DEV), pos))


def test_combine_gradients_by_differences():
    """Small whole numbers, for which every sum is exact: the gradients are the
    differences that one step of an input makes, to the bit."""
    T, k, E, H = 5, 3, 4, 16
    g = torch.Generator().manual_seed(3)
    ints = lambda *s: torch.randint(-4, 5, s, generator=g).float().to(DEV)  # noqa: E731
    _, _, pos = B.qmoe_sort_experts(dev(ids_of(T, k, E, 2, 0.2)), E)
    x, ys, w, dout, res = ints(T, H), ints(T * k, H), ints(T, k), ints(T, H), ints(T, H)
    dys, dw = B.qmoe_combine_backward(dout, ys, pos, w, dys=torch.zeros_like(ys))
    loss = lambda y, v: float((dout.double() * B.qmoe_combine(y, pos, v, res).double()).sum())  # noqa: E731
    base = loss(ys, w)
    for t, grad in ((ys, dys), (w, dw)):
        for i in range(0, t.numel(), 7 if t is ys else 1):
            up = t.clone()
            up.view(-1)[i] += 1
            assert (loss(up, w) if t is ys else loss(ys, up)) - base == float(grad.reshape(-1)[i])
    dxs = ints(T * k, H)
    dx = B.qmoe_dispatch_backward(dxs, pos)
    there = lambda v: float((dxs.double() * B.qmoe_dispatch(v, pos, out=torch.zeros_like(dxs)).double()).sum())  # noqa: E731
    for i in range(0, x.numel(), 5):
        up = x.clone()
        up.view(-1)[i] += 1
        assert there(up) - there(x) == float(dx.view(-1)[i])


def test_large_offsets():
    """More than 2^32 bytes: rows at the far end are read and written where they are."""
    T, k, H = 80000, 4, 8192
    x = torch.zeros((T, H), dtype=F16, device=DEV)
    tail = make(50, H, 5, F16).to(DEV)
    x[-50:] = tail
    pos = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
    pos[-50:] = torch.arange(T * k - 200, T * k, device=DEV, dtype=torch.int32).view(50, 4)
    xs = torch.empty((T * k, H), dtype=F16, device=DEV)
    B.qmoe_dispatch(x, pos, out=xs)
    assert torch.equal(xs[-200:], tail.repeat_interleave(4, 0))
    codes, scales = torch.empty((T * k, H), dtype=torch.uint8, device=DEV), torch.empty((T * k, H // 128), device=DEV)
    B.qmoe_fp8_quantize(x, pos, codes=codes, scales=scales)
    c, s = B.qmoe_fp8_quantize(tail)
    assert torch.equal(codes[-200:], c.repeat_interleave(4, 0)) and torch.equal(scales[-200:], s.repeat_interleave(4, 0))
    out = B.qmoe_combine(xs, pos)
    assert torch.equal(out[-50:], 4 * tail) and not out[:1000].any()
    dys, dw = B.qmoe_combine_backward(x, xs, pos, dys=xs)
    assert torch.equal(dys[-200:], tail.repeat_interleave(4, 0)) and not dw[:-50].any() and dw[-50:].all()
    # the product reads rows and writes outputs beyond 2^32 bytes
    wc, ws = B.qmoe_fp8_quantize_weights(make(64, H, 6, F16, 0.0).to(DEV))
    off = torch.tensor([T * k - 200, T * k], dtype=torch.int32, device=DEV)
    y = B.qmoe_fp8_matmul(codes, scales, wc[None], ws[None], F16, offsets=off)
    # (within the bound: how K is split, and so the order of the sums, goes by the number of rows)
    check_product((codes[-200:].cpu().numpy(), scales[-200:].cpu().numpy(), wc.cpu().numpy()[None], ws.cpu().numpy()[None]), y[-200:], F16)


# ---------------------------------------------------------------- the layer
def layer(x, rw, gu, down, k, residual):
    tw, ids, _, _ = B.qmoe_route(x, rw, k)
    E = rw.shape[1]
    off, perm, pos = B.qmoe_sort_experts(ids, E)
    h = B.qmoe_fp8_matmul(*B.qmoe_fp8_quantize(x, pos), *gu, x.dtype, offsets=off)
    y = B.qmoe_fp8_matmul(*B.qmoe_fp8_quantize_swiglu(h), *down, x.dtype, offsets=off)
    return B.qmoe_combine(y, pos, tw, residual), (tw, ids, off, perm, pos, h, y)


@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 128, 8, 2), (37, 256, 144, 8, 2), (200, 512, 256, 60, 4)])
def test_layer_of_fp8_experts(T, H, I, E, k):
    """The operators together, against a plain layer in 64 bits with the quantised
    weights and each stage's own input; then captured, with new tokens replayed."""
    g = torch.Generator(device=DEV).manual_seed(T)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    x, rw, res = rnd(T, H).bfloat16(), (0.1 * rnd(H, E)).bfloat16(), rnd(T, H).bfloat16()
    gu, down = B.qmoe_fp8_quantize_weights(H ** -0.5 * rnd(E, 2 * I, H)), B.qmoe_fp8_quantize_weights(I ** -0.5 * rnd(E, H, I))
    out, (tw, ids, off, perm, pos, h, y) = layer(x, rw, gu, down, k, res)
    W = lambda p: np.stack([fp8.values(c, s, 128) for c, s in zip(p[0].cpu().numpy(), p[1].cpu().numpy())])  # noqa: E731
    offs, Wg, Wd = off.cpu().numpy(), W(gu), W(down)
    tok = perm.cpu().numpy() // k
    X = fp8.values(*fp8.quantize(f64(x)))[tok]
    ref, mag = fp8.product(X, Wg, offs)
    assert (np.abs(f64(h) - ref) <= bound_of(ref, mag, H, BF16)).all()
    # SwiGLU's codes may fall on either side of a border: its own codes are checked above
    c, s = B.qmoe_fp8_quantize_swiglu(h)
    A = fp8.values(c.cpu().numpy(), s.cpu().numpy())
    assert (np.abs(A - fp8.swiglu(f64(h))) <= 2.0 ** -4 * (1 + 2.0 ** -19) * np.abs(A) + np.repeat(f64(s), 128, 1)[:, :I] * 2.0 ** -10).all()
    ref, mag = fp8.product(A, Wd, offs)
    assert (np.abs(f64(y) - ref) <= bound_of(ref, mag, I, BF16)).all()
    ref, mag = fp8.combine(f64(y), pos.cpu().numpy(), f64(tw), f64(res))
    assert (np.abs(f64(out) - ref) <= (k + 2) * 2.0 ** -24 * mag + 2.0 ** -8 * np.abs(ref)).all()
    # gradients of the way back, as a router's training wants them
    dout = rnd(T, H).bfloat16()
    dy, dw = B.qmoe_combine_backward(dout, y, pos, tw)
    rys, rw_, mag = fp8.combine_backward(f64(dout), f64(y), pos.cpu().numpy(), f64(tw))
    assert (np.abs(f64(dy) - rys) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(rys) + 1e-38).all() and (np.abs(f64(dw) - rw_) <= H * 2.0 ** -24 * mag).all()
    ws = B.Workspace(T, H, 32, E, k)
    tokens = x.clone()
    B._check(0, "")
    graph = torch.cuda.CUDAGraph()

    def step():
        tw, ids, _, _ = B.qmoe_route(tokens, rw, k, ws=ws)
        o, _, p = B.qmoe_sort_experts(ids, E)
        h = B.qmoe_fp8_matmul(*B.qmoe_fp8_quantize(tokens, p), *gu, BF16, offsets=o)
        return B.qmoe_combine(B.qmoe_fp8_matmul(*B.qmoe_fp8_quantize_swiglu(h), *down, BF16, offsets=o), p, tw, res)
    with torch.cuda.graph(graph):
        got = step()
    for seed in range(3):
        tokens.copy_(torch.randn((T, H), generator=g, device=DEV))
        graph.replay()
        assert torch.equal(got, layer(tokens, rw, gu, down, k, res)[0])


def test_gradient_with_respect_to_x_is_a_product_with_the_transposed_weights():
    """128 x 128 blocks transpose as they are."""
    N, K, M = 256, 384, 40
    g = torch.Generator().manual_seed(1)
    w = torch.randn((N, K), generator=g)
    wc, ws = B.qmoe_fp8_quantize_weights(w.to(DEV))
    tc, ts = B.qmoe_fp8_quantize_weights(w.t().contiguous().to(DEV))
    assert torch.equal(tc, wc.t()) and torch.equal(ts, ws.t())
    dy = make(M, N, 2, BF16, 0.0)
    dx = B.qmoe_fp8_matmul(*B.qmoe_fp8_quantize(dy.to(DEV)), tc, ts, F32)
    dyv = fp8.values(*fp8.quantize(f64(dy)))
    W = fp8.values(wc.cpu().numpy(), ws.cpu().numpy(), 128)
    ref, mag = dyv @ W, np.abs(dyv) @ np.abs(W)
    assert (np.abs(f64(dx) - ref) <= bound_of(ref, mag, N, F32)).all()


def test_first_calls_of_a_process_inside_a_capture():
    """Nothing of the operators needs a call before the capture."""
    code = """
import sys; sys.path.insert(0, %r)
import torch
from int4_block_quantized_gb300 import binding as B
g = torch.Generator(device="cuda").manual_seed(1)
x, w = torch.randn((9, 512), generator=g, device="cuda").half(), torch.randn((4, 512, 512), generator=g, device="cuda").half()
ids = torch.randint(0, 4, (9, 2), generator=g, device="cuda", dtype=torch.int32)
tw = torch.rand((9, 2), generator=g, device="cuda")
def run():
    off, perm, pos = B.qmoe_sort_experts(ids, 4)
    h = B.qmoe_fp8_matmul(*B.qmoe_fp8_quantize(x, pos), *B.qmoe_fp8_quantize_weights(w), torch.float16, offsets=off)
    c, s = B.qmoe_fp8_quantize_swiglu(h)
    y = B.qmoe_dispatch(x, pos)
    return (off, perm, pos, h, B.qmoe_fp8_dequant(c, s), B.qmoe_combine(y, pos, tw, x)) + B.qmoe_combine_backward(x, y, pos, tw)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = run()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, run()))
""" % ROOT
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300)
