"""The gradient of a grouped FP8 product with respect to its tokens: a product with
each expert's transposed codes and scales."""
import numpy as np
import pytest
import torch

from int4_block_quantized_gb300 import binding as B
from oracle import fp8

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32 = torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int4_block_quantized_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def f64(t):
    return t.detach().cpu().double().numpy()


@pytest.mark.parametrize("E,N,K,counts", [(3, 144, 272, (5, 0, 40)), (2, 400, 144, (130, 1)), (4, 16, 1424, (1, 2, 3, 4)), (1, 272, 400, (300,))])
def test_gradient_of_a_grouped_product(E, N, K, counts):
    """dx of y = x W[e]^T, N and K off 128: codes and scales of each expert transposed.
    Tolerance: (128 + nb + 4) 2^-23 of the sum of magnitudes, as in test_gpu_fp8.py."""
    g = torch.Generator().manual_seed(N + K)
    wc, ws = B.qmoe_fp8_quantize_weights(torch.randn((E, N, K), generator=g).to(DEV))
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    M = int(off[-1]) + 3
    dyc, dys = B.qmoe_fp8_quantize(torch.randn((M, N), generator=g).to(DEV))
    tc, ts = wc.transpose(1, 2).contiguous(), ws.transpose(1, 2).contiguous()
    dx = B.qmoe_fp8_matmul(dyc, dys, tc, ts, F32, offsets=torch.from_numpy(off).to(DEV), out=torch.full((M, K), 7.0, device=DEV))
    W = np.stack([fp8.values(c, s, 128) for c, s in zip(wc.cpu().numpy(), ws.cpu().numpy())])
    ref, mag = fp8.product(fp8.values(dyc.cpu().numpy(), dys.cpu().numpy()), W.transpose(0, 2, 1), off)
    n = int(off[-1])
    bound = (128 + -(-N // 128) + 4) * 2.0 ** -23 * mag + 2.0 ** -24 * np.abs(ref)
    assert (np.abs(f64(dx) - ref) <= bound)[:n].all() and (dx[n:] == 7).all()
