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
