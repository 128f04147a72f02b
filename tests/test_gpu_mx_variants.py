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


# every form that mm_choose gives: (x, M, N, K, (tokens a tile, pair, CTAs along
# K, spread codes)); odd numbers of tokens, outputs a multiple of 8 (16-bit rows
# on 16 bytes) and not of 128; several tiles to a CTA or pair where K is not shared
VARIANTS = [
    (B.MXFP8, 1, 24, 128, (16, 0, 1, 0)), (B.MXFP8, 1, 5000, 3584, (16, 0, 2, 0)),
    (B.MXFP8, 1, 2480, 1536, (16, 0, 4, 0)), (B.MXFP8, 1, 24, 1408, (16, 0, 8, 0)),
    (B.MXFP8, 17, 24, 128, (32, 0, 1, 0)), (B.MXFP8, 24, 4968, 2048, (32, 0, 2, 0)),
    (B.MXFP8, 19, 2496, 1664, (32, 0, 4, 0)), (B.MXFP8, 17, 24, 1280, (32, 0, 8, 0)),
    (B.MXFP8, 5786, 520, 128, (64, 0, 1, 0)), (B.MXFP8, 2473, 24, 2560, (64, 0, 2, 0)),
    (B.MXFP8, 1288, 24, 1664, (64, 0, 4, 0)), (B.MXFP8, 34, 24, 1664, (64, 0, 8, 0)),
    (B.MXFP8, 4081, 1712, 128, (128, 0, 1, 0)), (B.MXFP8, 1828, 2512, 1024, (128, 0, 1, 0)),
    (B.MXFP8, 5057, 24, 6528, (128, 0, 2, 0)), (B.MXFP8, 2755, 24, 8320, (128, 0, 4, 0)),
    (B.MXFP8, 4552, 2064, 128, (192, 0, 1, 0)), (B.MXFP8, 1173, 4032, 896, (192, 0, 1, 0)),
    (B.MXFP8, 2117, 4336, 1280, (192, 1, 1, 0)), (B.MXFP8, 1003, 4888, 1280, (192, 1, 1, 0)),
    (B.MXFP8, 3288, 4256, 128, (256, 1, 1, 0)), (B.MXFP8, 3566, 2096, 896, (256, 1, 1, 0)),
    (B.MXFP8, 1, 24, 32, (16, 0, 1, 1)), (B.MXFP8, 1, 4896, 1984, (16, 0, 2, 1)),
    (B.MXFP8, 1, 2384, 1088, (16, 0, 4, 1)), (B.MXFP8, 1, 24, 1056, (16, 0, 8, 1)),
    (B.MXFP8, 17, 24, 32, (32, 0, 1, 1)), (B.MXFP8, 19, 4984, 1728, (32, 0, 2, 1)),
    (B.MXFP8, 17, 2496, 1056, (32, 0, 4, 1)), (B.MXFP8, 18, 24, 1056, (32, 0, 8, 1)),
    (B.MXFP8, 771, 4200, 32, (64, 0, 1, 1)), (B.MXFP8, 2441, 24, 1440, (64, 0, 2, 1)),
    (B.MXFP8, 1173, 24, 1056, (64, 0, 4, 1)), (B.MXFP8, 35, 24, 1056, (64, 0, 8, 1)),
    (B.MXFP8, 1581, 4448, 32, (128, 0, 1, 1)), (B.MXFP8, 606, 5064, 864, (128, 0, 1, 1)),
    (B.MXFP8, 4957, 24, 4128, (128, 0, 2, 1)), (B.MXFP8, 2459, 24, 4928, (128, 0, 4, 1)),
    (B.MXFP8, 4857, 1552, 32, (192, 0, 1, 1)), (B.MXFP8, 4484, 1048, 832, (192, 0, 1, 1)),
    (B.MXFP4, 1, 24, 32, (16, 0, 1, 0)), (B.MXFP4, 1, 4896, 4160, (16, 0, 2, 0)),
    (B.MXFP4, 1, 2448, 2592, (16, 0, 4, 0)), (B.MXFP4, 1, 24, 2336, (16, 0, 8, 0)),
    (B.MXFP4, 17, 24, 32, (32, 0, 1, 0)), (B.MXFP4, 23, 4896, 5792, (32, 0, 2, 0)),
    (B.MXFP4, 20, 2416, 2592, (32, 0, 4, 0)), (B.MXFP4, 17, 24, 2336, (32, 0, 8, 0)),
    (B.MXFP4, 617, 4952, 32, (64, 0, 1, 0)), (B.MXFP4, 385, 5224, 992, (64, 0, 1, 0)),
    (B.MXFP4, 2456, 24, 4448, (64, 0, 2, 0)), (B.MXFP4, 1238, 24, 2912, (64, 0, 4, 0)),
    (B.MXFP4, 33, 24, 2656, (64, 0, 8, 0)), (B.MXFP4, 2502, 2704, 32, (128, 0, 1, 0)),
    (B.MXFP4, 5060, 776, 864, (128, 0, 1, 0)), (B.MXFP4, 2593, 3608, 32, (192, 0, 1, 0)),
    (B.MXFP4, 814, 5704, 864, (192, 0, 1, 0)), (B.MXFP4, 3075, 2920, 2368, (192, 1, 1, 0)),
    (B.MXFP4, 810, 5744, 2400, (192, 1, 1, 0)), (B.MXFP4, 4815, 3032, 32, (256, 1, 1, 0)),
    (B.MXFP4, 1838, 4120, 832, (256, 1, 1, 0)),
]


@pytest.mark.parametrize("xf,M,N,K,variant", VARIANTS)
def test_every_variant(xf, M, N, K, variant):
    """The size runs the form that it is listed for, which is right with each way
    of writing y: 32 bits, 16-bit rows on 16 bytes, and 16 bits on any place."""
    x, w, xd, wd = make(M, N, K, xf, M + N)
    assert B.qmoe_mx_matmul_variant(xf, wd[0], M) == variant
    y = B.qmoe_mx_matmul(*xd, xf, *wd, torch.float32)
    check(x, xf, w, y)
    for dtype, at in ((torch.bfloat16, 64), (torch.float16, 64), (torch.float16, 33)):
        buf = torch.full((M * N + 128,), 7.0, dtype=dtype, device=DEV)
        out = B.qmoe_mx_matmul(*xd, xf, *wd, dtype, out=buf[at:at + M * N].view(M, N))
        assert torch.equal(out, y.to(dtype))  # the same sums, rounded once
        assert (buf[:at] == 7).all() and (buf[at + M * N:] == 7).all()


def test_every_variant_is_listed():
    """Sizes of all kinds run no form that the list leaves out."""
    listed = {(v[0], v[4]) for v in VARIANTS}
    rng = np.random.default_rng(0)
    w = torch.empty(6000 * 4096, dtype=torch.uint8, device=DEV)
    for _ in range(4000):
        M, N, nb = (int(np.exp(rng.uniform(0, np.log(n)))) for n in (6000, 6000, 256))
        wc = w[:N * nb * 16].view(N, nb * 16)
        for xf in (B.MXFP8, B.MXFP4):
            assert (xf, B.qmoe_mx_matmul_variant(xf, wc, M)) in listed, (xf, M, N, 32 * nb)


def test_pairs_beside_the_layer_on_another_stream():
    """The layer's tensor-core kernels (router, grouped GEMM) and pairs of CTAs
    each take tensor memory; on two streams at once both finish with their own results."""
    from int4_block_quantized_gb300 import synthetic as S
    wl = S.WORKLOADS["prefill"]
    layer = dict(S.make_layer(wl, seed=1, device=DEV))
    ws = B.Workspace(wl.T, wl.H, wl.I, wl.E, wl.k, device=DEV)
    _, w_ref, ids_ref = B.qmoe_forward(layer, ws=ws, return_routing=True)
    args = [make(M, N, K, xf, 3)[2:] + (xf,) for M, N, K, xf in (PAIRS[0], PAIRS[4])]
    assert all(B.qmoe_mx_matmul_variant(xf, w[0], x[0].shape[0])[1] == 1 for x, w, xf in args)
    refs = [B.qmoe_mx_matmul(*x, xf, *w) for x, w, xf in args]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got, routed = [], []
    for i in range(30):
        routed.append(B.qmoe_forward(layer, ws=ws, return_routing=True)[1:])
        with torch.cuda.stream(side):
            x, w, xf = args[i % 2]
            got.append(B.qmoe_mx_matmul(*x, xf, *w))
    torch.cuda.synchronize()
    assert ws.status() == (0, 0) and B.qmoe_mx_status() == (0, 0)
    assert all(torch.equal(w, w_ref) and torch.equal(i, ids_ref) for w, i in routed)
    assert all(torch.equal(y, refs[i % 2]) for i, y in enumerate(got))


def test_outputs_beyond_32_bit_offsets():
    """More than 2^32 outputs, whichever way they are written: the last tokens as
    computed alone (K = 32 is one instruction, so the sums are the same ones)."""
    M, N, K = 66001, 65608, 32
    x, w = random_mx(M, K, B.MXFP8, 1), random_mx(N, K, B.MXFP4, 2)
    wd = to_dev(*w, B.MXFP4)
    tail = to_dev(x[0][-300:], x[1][-300:], B.MXFP8)
    for dtype, n in ((torch.bfloat16, N), (torch.bfloat16, N - 1), (torch.float32, N)):
        wn = wd if n == N else to_dev(w[0][:n], w[1][:n], B.MXFP4)
        y = B.qmoe_mx_matmul(*to_dev(*x, B.MXFP8), B.MXFP8, *wn, dtype)
        assert torch.equal(y[-300:], B.qmoe_mx_matmul(*tail, B.MXFP8, *wn, dtype))
        del y
