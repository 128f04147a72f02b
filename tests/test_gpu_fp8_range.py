"""FP8 operators where fp32 runs out of exponents: SwiGLU's gates far below zero
beside a large `up`, and products whose scales leave fp32's range when they are
multiplied with each other."""
import numpy as np
import pytest
import torch

from int4_block_quantized_gb300 import binding as B
from oracle import fp8

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int4_block_quantized_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def f64(t):
    return t.detach().cpu().double().numpy()


# ----------------------------------------------------------------- SwiGLU
def check_swiglu(h):
    """Codes and scales as test_gpu_fp8.py derives them: a relative error of at most
    9 2^-24.  For gates far below zero that is the exponential's 2 units (4 2^-24),
    a constant's rounding and three products', 8 2^-24 in all; 1 + exp(gate) is 1."""
    I = h.shape[1] // 2
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


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lo,hi", [(-95, -85), (-130, -80), (-178, -96), (-90, 3)])
def test_swiglu_of_gates_far_below_zero(lo, hi, dtype):
    """exp(-gate) leaves fp32 from about -88.7 down, its reciprocal's normal numbers
    from -87.3: the product with a large `up` is a number all the same."""
    g = torch.Generator().manual_seed(lo * lo + hi)
    h = torch.empty((64, 2 * 272))
    h[:, :272] = lo + (hi - lo) * torch.rand((64, 272), generator=g)
    h[:, 272:] = torch.randn((64, 272), generator=g) * torch.exp2(60 + 64 * torch.rand((64, 1), generator=g))
    h[:8, 272:] *= 2.0 ** -50  # nothing left of these but where gates are near -90
    h[:, 5:272:31] = 0.25 * torch.randint(-356, -344, (64, 9), generator=g).float()  # -89 .. -86
    check_swiglu(h.clamp(-3e38, 3e38).to(dtype))


def test_swiglu_of_fp16_gates_far_below_zero():
    """The largest fp16 `up` keeps these above the least block maximum's codes."""
    g = torch.Generator().manual_seed(7)
    h = torch.empty((40, 2 * 144))
    h[:, :144] = -93 + 10 * torch.rand((40, 144), generator=g)
    h[:, 144:] = 65504 * (2 * torch.rand((40, 144), generator=g) - 1)
    h[0, :144] = -65504
    check_swiglu(h.to(F16))


def test_swiglu_of_gates_far_below_zero_leaves_others_alone():
    """Elements beside them get the bits that they get without them."""
    g = torch.Generator().manual_seed(8)
    h = 3 * torch.randn((32, 2 * 256), generator=g)
    h[:, 0] = h[:, 128] = 20  # the blocks' largest
    h[:, 256] = h[:, 256 + 128] = 30
    deep = h.clone()
    at = torch.rand((32, 256), generator=g) < 0.1
    at[:, 0] = at[:, 128] = False
    deep[:, :256][at] = -90.0
    (ca, sa), (cb, sb) = (B.qmoe_fp8_quantize_swiglu(v.to(DEV)) for v in (h, deep))
    assert torch.equal(sa, sb) and torch.equal(ca.cpu()[~at], cb.cpu()[~at]) and not (cb.cpu()[at] & 127).any()


# ----------------------------------------------------------------- product
# (M, N, K, experts or None): every tile of both forms, with K shared and not
SIZES = [(3, 8, 16, 2), (50, 1562, 448, None), (106, 8, 672, 2), (3, 8, 912, None), (143, 1, 16, 2), (99, 1491, 512, None), (136, 1, 432, 2),
         (150, 4, 976, 2), (132, 2, 16, None), (588, 397, 1424, None), (428, 70, 816, 3), (268, 28, 960, 2), (5714, 797, 80, None),
         (2165, 64, 4544, 60), (108, 2482, 3344, None), (963, 3, 3856, 8), (290, 8, 400, 2), (3604, 400, 384, 60), (900, 2561, 512, None),
         (4086, 607, 416, 2)]


def test_the_sizes_reach_every_tile():
    forms = [B.qmoe_fp8_matmul_variant(*s) for s in SIZES]
    assert {f[:2] for f in forms} == {(16, 0), (32, 0), (64, 0), (128, 0), (128, 1), (256, 1)} and {f[2] for f in forms} == {1, 2, 4, 8}


def operands(M, N, K, E):
    """(codes and scales, offsets or None); scales within 2^-6 .. 2^-4, not powers of two."""
    g = torch.Generator(device=DEV).manual_seed(M + N + K)
    nb, rb, n = -(-K // 128), -(-N // 128), E or 1

    def codes(*s):
        c = torch.randint(0, 256, s, generator=g, device=DEV, dtype=torch.int32)
        return torch.where(c & 127 == 127, c ^ 1, c).to(torch.uint8)

    def scales(*s):
        return torch.rand(s, generator=g, device=DEV) * 3 * 2.0 ** -6 + 2.0 ** -6
    off = None
    if E:
        cut = torch.sort(torch.randint(0, M + 1, (E - 1,), generator=g, device=DEV)).values.int()
        off = torch.cat((torch.zeros_like(cut[:1]), cut, torch.full_like(cut[:1], M)))
    return codes(M, K), scales(M, nb), codes(n, N, K), scales(n, rb, nb), off


def product(xc, xs, wc, ws, off, dtype):
    if off is None:
        wc, ws = wc[0], ws[0]
    out = torch.full((xc.shape[0], wc.shape[-2]), 7.0, dtype=dtype, device=DEV)
    return B.qmoe_fp8_matmul(xc, xs, wc, ws, dtype, offsets=off, out=out)


def check_product(y, xc, xs, wc, ws, off):
    """Within (128 + nb + 4) 2^-23 of the sum of magnitudes and one rounding of the
    result (as test_gpu_fp8.py derives it), below fp32's normal numbers within half a
    step there; what is beyond the largest number is infinite."""
    K, N = xc.shape[1], wc.shape[1]
    k, r = torch.arange(K, device=DEV) // 128, torch.arange(N, device=DEV) // 128
    X = xc.view(torch.float8_e4m3fn).double() * xs.double()[:, k]
    W = wc.view(torch.float8_e4m3fn).double() * ws.double()[:, r][:, :, k]
    f, nb = torch.finfo(y.dtype), xs.shape[1]
    ends = [0, xc.shape[0]] if off is None else off.tolist()
    for e in range(W.shape[0]):
        x, got = X[ends[e]:ends[e + 1]], y[ends[e]:ends[e + 1]].double()
        ref, mag = x @ W[e].T, x.abs() @ W[e].abs().T
        # sums in fp32 may end below its normal numbers: half a step of 2^-149 for each of the nb additions
        bound = (1 + f.eps) * (128 + nb + 4) * 2.0 ** -23 * mag + f.eps / 2 * ref.abs() + f.smallest_normal * f.eps / 2 + nb * 2.0 ** -150
        over = ref.abs() - bound > f.max
        assert torch.equal(got[over], torch.inf * ref[over].sign())
        fine = ref.abs() + bound <= f.max
        assert ((got - ref).abs() <= bound)[fine].all(), (e, float(((got - ref).abs() / bound)[fine].max()))


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("tokens,weights", [(-64, -64), (-69, -69), (-134, 20), (30, -143), (-110, -40)])
def test_scales_whose_product_is_below_fp32(size, tokens, weights):
    """Every other token's scales times 2^tokens, all weights' times 2^weights: the
    product has lost bits in fp32 (or all of them), what it gives with the codes' sum
    has not.  The tokens between have scales that bring the product back, and get the
    bits that they get beside ordinary tokens."""
    xc, xs, wc, ws, off = operands(*size)
    ws = ws * 2.0 ** weights
    plain = xs * 2.0 ** min(max(-weights, 0), 100)
    odd = plain.clone()
    odd[::2] = xs[::2] * 2.0 ** tokens
    for dtype in (F32, BF16):
        y = product(xc, odd, wc, ws, off, dtype)
        check_product(y, xc, odd, wc, ws, off)
        assert torch.equal(y[1::2], product(xc, plain, wc, ws, off, dtype)[1::2])


@pytest.mark.parametrize("size", SIZES)
def test_scales_whose_product_is_above_fp32(size):
    """Products from 2^128 on: a sum of 0 gives 0, a small one a number, others
    infinity; the tokens between are ordinary."""
    xc, xs, wc, ws, off = operands(*size)
    ws, odd = ws * 2.0 ** 70, xs * 2.0 ** -70
    plain = odd.clone()
    odd[::2] = xs[::2] * 2.0 ** 70
    xc[::2] = 0
    xc[::4, 3] = 1     # 2^-9 in the first block
    xc[8::16, 3] = 0x81  # and its negative
    for dtype in (F32, BF16):
        y = product(xc, odd, wc, ws, off, dtype)
        check_product(y, xc, odd, wc, ws, off)
        assert not y[2::4].any() and torch.equal(y[1::2], product(xc, plain, wc, ws, off, dtype)[1::2])


@pytest.mark.parametrize("size", [s for s in SIZES if s[2] > 128])
def test_one_block_of_one_token_out_of_range(size):
    """All of the token's other blocks are 0; nobody else's bits change, with scales of
    either sign and some that are 0."""
    xc, xs, wc, ws, off = operands(*size)
    xs[::3] *= -1
    ws[:, :, 1::2] *= -1
    xs[-1] = 0
    ref = product(xc, xs, wc, ws, off, F32)
    check_product(ref, xc, xs, wc, ws, off)
    m, b = size[0] // 2, (size[2] - 1) // 256
    odd, xc2 = xs.clone(), xc.clone()
    odd[m, b] = odd[m, b] * 2.0 ** -128
    xc2[m] = 0
    xc2[m, 128 * b:128 * b + 128] = xc[m, 128 * b:128 * b + 128]
    y = product(xc2, odd, wc, ws, off, F32)
    check_product(y, xc2, odd, wc, ws, off)
    assert y[m].any() and torch.equal(y[:m], ref[:m]) and torch.equal(y[m + 1:], ref[m + 1:])


@pytest.mark.parametrize("M,E", [(5, None), (300, None), (700, 3)])
def test_infinite_and_nan_scales_stay_where_they_enter(M, E):
    """An infinite scale times a sum of 0 is NaN, times another infinite; a NaN is NaN;
    neither touches other tokens."""
    xc, xs, wc, ws, off = operands(M, 200, 400, E)
    ref = product(xc, xs, wc, ws, off, F32)
    odd = xs.clone()
    odd[0, 1], odd[2, 0], odd[3, 3], xc2 = torch.inf, torch.nan, -torch.inf, xc.clone()
    xc2[3, 384:] = 0
    y = product(xc2, odd, wc, ws, off, F32)
    assert torch.isinf(y[0]).any() and not torch.isfinite(y[0]).any() and torch.isnan(y[2:4]).all()
    assert torch.equal(y[1], ref[1]) and torch.equal(y[4:], ref[4:])
