"""The product's bounded waits run to expiry: one of its roles waits for an
arrival that nothing makes, under a limit of 2^20 SM cycles (about 0.5 ms).
Every role drains and returns, the status word reads the time-out, and the
next call on the same tensors computes the same bits as before."""
import numpy as np
import pytest
import torch

from int4_block_quantized_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
LIMIT = 1024  # x 1024 SM cycles


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int4_block_quantized_gb300 import build
    build.build()
    assert torch.cuda.is_available()


# one CTA a tile; K over 8 CTAs, all of it in the ring at once; over 2, the
# ring taking the sums; several tiles a CTA; pairs, both kinds; spread codes
SHAPES = {"one": (40, 300, 128, 0), "split": (1, 1408, 2048, 0), "split in the ring": (471, 1465, 4288, 0),
          "tiles": (2600, 1912, 256, 0), "pairs of 192": (1679, 2710, 1280, 0), "pairs of 256": (5321, 1313, 256, 1),
          "spread": (300, 2000, 1440, 0), "spread, split": (18, 130, 2912, 0), "4 bits": (20, 700, 2400, 1)}


def tensors(M, N, K, xf):
    g = torch.Generator().manual_seed(M)
    x = B.qmoe_mx_quantize(torch.randn((M, K), generator=g).to(DEV), xf)
    return x, B.qmoe_mx_quantize(torch.randn((N, K), generator=g).to(DEV), B.MXFP4)


def run_out(x, xf, w, flags, **kw):
    """(status bits, seconds on the device, y) of a call that stalls."""
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    a.record()
    y = B.qmoe_mx_matmul(*x, xf, *w, torch.bfloat16, status=status, diagnostics=(LIMIT, flags), **kw)
    b.record()
    torch.cuda.synchronize()
    return int(status.item()), a.elapsed_time(b) * 1e-3, y


@pytest.mark.parametrize("name", ["one", "split", "tiles", "pairs of 192", "pairs of 256", "4 bits"])
def test_a_stalled_mma_is_reported(name):
    M, N, K, xf = SHAPES[name]
    x, w = tensors(M, N, K, xf)
    ref = B.qmoe_mx_matmul(*x, xf, *w)
    assert run_out(x, xf, w, B.DIAG_STALL_MX_MMA)[0] == 1
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for diagnostics in (None, (0, 0)):
        assert torch.equal(B.qmoe_mx_matmul(*x, xf, *w, status=status, diagnostics=diagnostics), ref)
    assert int(status.item()) == 0


ROLES = {"codes": B.DIAG_STALL_MX_CODES, "scales": B.DIAG_STALL_MX_SCALES, "mma": B.DIAG_STALL_MX_MMA,
         "output": B.DIAG_STALL_MX_OUTPUT, "spread": B.DIAG_STALL_MX_SPREAD}


SPREADS = ("spread", "spread, split", "split in the ring")  # the sizes whose codes are spread


@pytest.mark.parametrize("name,role", [(n, r) for n in SHAPES for r in ROLES if r != "spread" or n in SPREADS])
def test_a_stalled_role_drains_against_one_deadline(name, role):
    """However many slots are in flight, and whichever role it is: the limit of
    0.5 ms and the 10 ms that copies get, not 2 s per slot.  Every CTA of a grid
    runs at once, so a second is generous."""
    M, N, K, xf = SHAPES[name]
    x, w = tensors(M, N, K, xf)
    ref = B.qmoe_mx_matmul(*x, xf, *w)
    bits, seconds, _ = run_out(x, xf, w, ROLES[role])
    assert bits == 1 and seconds < 1.0, seconds
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert torch.equal(B.qmoe_mx_matmul(*x, xf, *w, status=status), ref) and int(status.item()) == 0


def test_a_call_without_a_status_word_is_reported_too():
    """In the library's own word: read once, then clear; a call with a word of
    its own does not set it, and a captured call does."""
    M, N, K, xf = SHAPES["split"]
    x, w = tensors(M, N, K, xf)
    assert B.qmoe_mx_status() == (0, 0)
    B.qmoe_mx_matmul(*x, xf, *w, diagnostics=(LIMIT, B.DIAG_STALL_MX_MMA))
    assert B.qmoe_mx_status() == (5, 1)
    assert B.qmoe_mx_status() == (0, 0)
    assert run_out(x, xf, w, B.DIAG_STALL_MX_MMA)[0] == 1 and B.qmoe_mx_status() == (0, 0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.qmoe_mx_matmul(*x, xf, *w, diagnostics=(LIMIT, B.DIAG_STALL_MX_MMA))
    assert B.qmoe_mx_status() == (0, 0)
    g.replay()
    assert B.qmoe_mx_status() == (5, 1)
    B.qmoe_mx_matmul(*x, xf, *w)
    assert B.qmoe_mx_status() == (0, 0)
