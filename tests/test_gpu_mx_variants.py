"""GPU parity of the product's tile variants: the kernels that large products
run on, at the smallest sizes that reach them.

The tolerance is derived as in test_gpu_mx.py: products of two elements are
exact in fp32; a sum of K of them in any order, each addition off by at most a
whole step, is off by at most K 2^-23 times the sum of magnitudes, and the
result is rounded once (half a step of the output's type)."""
import numpy as np
import pytest
import torch

from int4_block_quantized_gb300 import binding as B
from oracle import mx

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int4_block_quantized_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def random_mx(R, K, fmt, seed):
    """(per-element codes, row-major scales) without NaN codes."""
    rng = np.random.default_rng(seed)
    c = rng.integers(0, 256 if fmt == B.MXFP8 else 16, (R, K)).astype(np.uint8)
    if fmt == B.MXFP8:
        c = np.where((c & 127) == 127, c ^ 1, c).astype(np.uint8)
    return c, rng.integers(112, 124, (R, K // 32)).astype(np.uint8)


def to_dev(c, s, fmt):
    return (torch.from_numpy(np.ascontiguousarray(mx.pack(c, fmt))).to(DEV),
            B.qmoe_mx_tile_scales(torch.from_numpy(s).to(DEV)))


def check(x, xf, w, y):
    """y against fp64 products of the values that codes and scales stand for."""
    X = torch.from_numpy(mx.values(*x, xf)).to(DEV)
    W = torch.from_numpy(mx.values(*w, B.MXFP4)).to(DEV)
    ref, mag = X @ W.T, X.abs() @ W.abs().T
    f = torch.finfo(y.dtype)
    bound = (1 + f.eps) * X.shape[1] * 2.0 ** -23 * mag + f.eps / 2 * ref.abs() + f.smallest_normal * f.eps / 2
    err = (y.double() - ref).abs()
    assert (err <= bound).all(), "worst %.3g of its bound" % float((err / bound).max())


def make(M, N, K, xf, seed):
    x, w = random_mx(M, K, xf, seed), random_mx(N, K, B.MXFP4, seed + 1)
    return x, w, to_dev(*x, xf), to_dev(*w, B.MXFP4)


# pairs of CTAs: 192 tokens a tile (two whole accumulators) and 256 (overlapping
# ones), several tiles to a pair, odd numbers of row and token tiles
PAIRS = [(1679, 2710, 1280, B.MXFP8), (4899, 919, 2048, B.MXFP8), (939, 4920, 2496, B.MXFP4),
         (4913, 683, 128, B.MXFP8), (5321, 1313, 256, B.MXFP8), (5321, 1313, 256, B.MXFP4), (779, 4531, 32, B.MXFP4)]


@pytest.mark.parametrize("M,N,K,xf", PAIRS)
def test_pairs(M, N, K, xf):
    """Right, and the same bits in launches that follow one another at once: the
    next one's CTAs take over each SM as soon as a pair has left it."""
    x, w, xd, wd = make(M, N, K, xf, M)
    outs = [B.qmoe_mx_matmul(*xd, xf, *wd, torch.float32) for _ in range(8)]
    check(x, xf, w, outs[0])
    assert all(torch.equal(o, outs[0]) for o in outs)
