"""Every form of the FP8 product (asked of qmoe_fp8_matmul_variant, so that a
refitted choice cannot move the sizes off their forms unnoticed) against fp64, and
its bounded waits run to expiry: a role waits for an arrival that nothing makes,
under a limit of 2^20 SM cycles (about 0.5 ms); every role drains and returns, the
status word reads the time-out, and the next call computes the same bits as before.

The tolerance is derived as in test_gpu_fp8.py: (128 + nb + 4) 2^-23 times the sum
of magnitudes for nb blocks of 128 k, and one rounding of the result."""
import numpy as np
import pytest
import torch

from int4_block_quantized_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
LIMIT = 1024  # x 1024 SM cycles

# (M, N, K, experts or None, (tile, form, CTAs along K)): odd numbers of tokens,
# outputs and blocks, several tiles to a CTA where K is not shared
FORMS = [
    (3, 8, 16, 2, (16, 0, 1)), (50, 1562, 448, None, (16, 0, 2)), (42, 2, 720, 60, (16, 0, 2)), (3, 1, 528, None, (16, 0, 4)),
    (106, 8, 672, 2, (16, 0, 4)), (3, 8, 912, None, (16, 0, 8)), (3, 1, 1056, 3, (16, 0, 8)), (67, 1, 16, None, (32, 0, 1)),
    (143, 1, 16, 2, (32, 0, 1)), (99, 1491, 512, None, (32, 0, 2)), (490, 353, 1392, 8, (32, 0, 2)),
    (76, 2, 416, None, (32, 0, 4)), (67, 1425, 2816, None, (32, 0, 4)), (136, 1, 432, 2, (32, 0, 4)),
    (69, 1, 1120, None, (32, 0, 8)), (150, 4, 976, 2, (32, 0, 8)), (132, 2, 16, None, (64, 0, 1)), (288, 8, 16, 2, (64, 0, 1)),
    (588, 397, 1424, None, (64, 0, 2)), (555, 2, 3152, 60, (64, 0, 2)), (188, 46, 832, None, (64, 0, 4)),
    (428, 70, 816, 3, (64, 0, 4)), (143, 1, 976, None, (64, 0, 8)), (268, 28, 960, 2, (64, 0, 8)),
    (5714, 797, 80, None, (128, 0, 1)), (4933, 261, 32, 60, (128, 0, 1)), (2165, 64, 4544, 60, (128, 0, 2)),
    (108, 2482, 3344, None, (128, 0, 4)), (160, 1328, 1696, 2, (128, 0, 4)), (88, 1848, 2928, None, (128, 0, 8)),
    (963, 3, 3856, 8, (128, 0, 8)), (137, 2, 416, None, (128, 1, 1)), (290, 8, 400, 2, (128, 1, 1)),
    (3604, 400, 384, 60, (128, 1, 1)), (900, 2561, 512, None, (256, 1, 1)), (1385, 1896, 1024, None, (256, 1, 1)),
    (4086, 607, 416, 2, (256, 1, 1)), (3262, 776, 992, 3, (256, 1, 1)), (3, 8, 400, 2, (16, 0, 4)), (65, 8, 960, None, (32, 0, 8)),
    (132, 8, 992, None, (64, 0, 8))]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int4_block_quantized_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def make(M, N, K, E, seed=0):
    """(operands, offsets or None, fp64 values x, w) on the device; an expert's rows
    are unequal, one has none, and the last rows belong to nobody."""
    g = torch.Generator().manual_seed(seed + M + N + K)
    nb, rb, n = -(-K // 128), -(-N // 128), E or 1

    def codes(*s):
        c = torch.randint(0, 256, s, generator=g, dtype=torch.int32)
        return torch.where(c & 127 == 127, c ^ 1, c).to(torch.uint8).to(DEV)

    def scales(*s):
        return (torch.rand(s, generator=g) * 2.0 ** -4 + 2.0 ** -6).to(DEV)
    ops = codes(M, K), scales(M, nb), codes(n, N, K), scales(n, rb, nb)
    k, r = torch.arange(K, device=DEV) // 128, torch.arange(N, device=DEV) // 128
    X = ops[0].view(torch.float8_e4m3fn).double() * ops[1].double()[:, k]
    W = ops[2].view(torch.float8_e4m3fn).double() * ops[3].double()[:, r][:, :, k]
    off = None
    if E is None:
        ops = ops[0], ops[1], ops[2][0], ops[3][0]
    else:
        cut = torch.sort(torch.randint(0, M + 1, (E - 1,), generator=g)).values
        cut[E // 2:E // 2 + 1] = cut[max(E // 2 - 1, 0)]
        off = torch.cat((torch.zeros(1, dtype=torch.long), cut, torch.tensor([M - M // 20]))).clamp(max=M - M // 20).int().to(DEV)
    return ops, off, X, W


def check(y, off, X, W):
    K, ends = X.shape[1], [0, X.shape[0]] if off is None else off.tolist()
    f = torch.finfo(y.dtype)
    for e in range(len(ends) - 1):
        x, got = X[ends[e]:ends[e + 1]], y[ends[e]:ends[e + 1]].double()
        ref, mag = x @ W[e].T, x.abs() @ W[e].abs().T
        bound = (1 + f.eps) * (128 + -(-K // 128) + 4) * 2.0 ** -23 * mag + f.eps / 2 * ref.abs() + f.smallest_normal * f.eps / 2
        assert ((got - ref).abs() <= bound).all(), (e, float(((got - ref).abs() / bound).max()))


@pytest.mark.parametrize("M,N,K,E,form", FORMS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_each_form(M, N, K, E, form, dtype):
    """Right, rows of nobody untouched, and the same bits in launches that follow
    one another at once."""
    assert B.qmoe_fp8_matmul_variant(M, N, K, E) == form
    ops, off, X, W = make(M, N, K, E)
    outs = [torch.full((M, N), 7.0, dtype=dtype, device=DEV) for _ in range(6)]
    for o in outs:
        B.qmoe_fp8_matmul(*ops, dtype, offsets=off, out=o)
    check(outs[0], off, X, W)
    assert all(torch.equal(o, outs[0]) for o in outs)
    if off is not None:
        assert (outs[0][int(off[-1]):] == 7).all()


@pytest.mark.parametrize("M,N,K,E,form", [(8192, 4900, 16, 256, (64, 0, 1)), (20000, 8199, 144, None, (128, 0, 1)),
                                          (20000, 8199, 272, None, (128, 1, 1)), (20000, 16000, 400, None, (256, 1, 1))])
def test_more_tiles_than_a_cta_lists(M, N, K, E, form):
    """Above 64 tiles to each of 152 CTAs: the first ones come from the list, the
    others are worked out by each role."""
    assert B.qmoe_fp8_matmul_variant(M, N, K, E) == form
    tiles = (E if E else -(-M // (128 if form[1] else form[0]))) * -(-N // (form[0] if form[1] else 128))
    assert tiles > 64 * 152
    ops, off, X, W = make(M, N, K, E)
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV)
    B.qmoe_fp8_matmul(*ops, offsets=off, out=y)
    check(y, off, X, W)
    if off is not None:
        assert (y[int(off[-1]):] == 7).all()


@pytest.mark.parametrize("K", [16, 400])
def test_more_than_2_to_the_32_outputs(K):
    M, N = 70000, 62000
    ops, _, X, W = make(M, N, K, None)
    y = B.qmoe_fp8_matmul(*ops)
    for m in (0, M // 2, M - 200):
        check(y[m:m + 200], None, X[m:m + 200], W)


def run_out(ops, off, flags):
    """(status bits, seconds on the device) of a call that stalls."""
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    a.record()
    B.qmoe_fp8_matmul(*ops, torch.bfloat16, offsets=off, status=status, diagnostics=(LIMIT, flags))
    b.record()
    torch.cuda.synchronize()
    return int(status.item()), a.elapsed_time(b) * 1e-3


ROLES = {"codes": B.DIAG_STALL_FP8_CODES, "scales": B.DIAG_STALL_FP8_SCALES, "mma": B.DIAG_STALL_FP8_MMA,
         "output": B.DIAG_STALL_FP8_OUTPUT}


@pytest.mark.parametrize("M,N,K,E,form", FORMS)
@pytest.mark.parametrize("role", ROLES)
def test_a_stalled_role_drains(M, N, K, E, form, role):
    """Whichever role it is: the limit of 0.5 ms and the 10 ms that copies get, not
    2 s per slot.  Every CTA of a grid runs at once, so a second is generous."""
    ops, off, _, _ = make(M, N, K, E)
    zeros = lambda: torch.zeros((M, N), dtype=torch.bfloat16, device=DEV)  # noqa: E731
    ref = B.qmoe_fp8_matmul(*ops, offsets=off, out=zeros())
    bits, seconds = run_out(ops, off, ROLES[role])
    assert bits == 1 and seconds < 1.0, seconds
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for diagnostics in (None, (0, 0)):
        assert torch.equal(B.qmoe_fp8_matmul(*ops, offsets=off, out=zeros(), status=status, diagnostics=diagnostics), ref)
    assert int(status.item()) == 0


def test_a_call_without_a_status_word_is_reported_too():
    """In the library's own word: read once, then clear; a call with a word of its
    own does not set it, and a captured call does."""
    ops, off, _, _ = make(40, 300, 512, None)
    assert B.qmoe_fp8_status() == (0, 0)
    stall = (LIMIT, B.DIAG_STALL_FP8_MMA)
    B.qmoe_fp8_matmul(*ops, diagnostics=stall)
    assert B.qmoe_fp8_status() == (5, 1) and B.qmoe_fp8_status() == (0, 0)
    assert run_out(ops, off, B.DIAG_STALL_FP8_MMA)[0] == 1 and B.qmoe_fp8_status() == (0, 0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.qmoe_fp8_matmul(*ops, diagnostics=stall)
    assert B.qmoe_fp8_status() == (0, 0)
    g.replay()
    assert B.qmoe_fp8_status() == (5, 1)
    B.qmoe_fp8_matmul(*ops)
    assert B.qmoe_fp8_status() == (0, 0)
