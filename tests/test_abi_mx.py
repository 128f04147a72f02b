"""Host-side checks of the microscaled entry points (no GPU): sizes, and bad
arguments refused with the documented status before anything is enqueued."""
import pytest
import torch

FAKE = 0x10000  # 16-byte aligned, never dereferenced: every call below fails its checks first


@pytest.fixture(scope="module")
def L():
    from int4_block_quantized_gb300 import build as b
    b.build()
    from int4_block_quantized_gb300 import binding
    return binding.lib()


def test_scale_bytes(L):
    assert L.qmoe_mx_scale_bytes(1, 32) == 512
    assert L.qmoe_mx_scale_bytes(128, 128) == 512
    assert L.qmoe_mx_scale_bytes(129, 160) == 4 * 512
    assert L.qmoe_mx_scale_bytes(2 ** 31 - 1, 2 ** 20) == 2 ** 24 * 2 ** 13 * 512
    for R, K in ((0, 32), (1, 0), (1, 48), (-1, 32), (1, -32)):
        assert L.qmoe_mx_scale_bytes(R, K) == 0


@pytest.mark.parametrize("kw", [dict(x=None), dict(x=FAKE + 8), dict(xdt=3), dict(xdt=-1), dict(fmt=2), dict(fmt=-1),
                                dict(M=0), dict(K=0), dict(K=48), dict(c=None), dict(c=FAKE + 4), dict(s=None),
                                dict(s=FAKE + 8)])
def test_quantize_and_dequant_refuse(L, kw):
    a = dict(x=FAKE, xdt=0, fmt=0, M=4, K=64, c=FAKE, s=FAKE)
    a.update(kw)
    assert L.qmoe_mx_quantize(a["x"], a["xdt"], a["fmt"], a["M"], a["K"], a["c"], a["s"], None) == 1
    assert L.qmoe_mx_dequant(a["c"], a["s"], a["fmt"], a["M"], a["K"], a["x"], a["xdt"], None) == 1


@pytest.mark.parametrize("kw", [dict(x=None), dict(x=FAKE + 8), dict(r=FAKE + 2), dict(w=FAKE + 4), dict(ro=FAKE + 8),
                                dict(dt=2), dict(eps=-1.0), dict(eps=float("nan")), dict(fmt=7), dict(T=0), dict(H=40),
                                dict(c=None), dict(s=None)])
def test_rmsnorm_refuses(L, kw):
    a = dict(x=FAKE, r=FAKE, w=FAKE, dt=0, T=4, H=64, eps=1e-6, fmt=0, ro=FAKE, c=FAKE, s=FAKE)
    a.update(kw)
    assert L.qmoe_rmsnorm_mx(a["x"], a["r"], a["w"], a["dt"], a["T"], a["H"], a["eps"], a["fmt"], a["ro"], a["c"],
                             a["s"], None) == 1


@pytest.mark.parametrize("kw", [dict(xc=None), dict(xs=None), dict(wc=None), dict(ws=None), dict(xc=FAKE + 8),
                                dict(xs=FAKE + 8), dict(wc=FAKE + 8), dict(ws=FAKE + 8), dict(fmt=2), dict(M=0),
                                dict(N=0), dict(K=0), dict(K=100), dict(y=None), dict(ydt=3), dict(y=FAKE + 1),
                                dict(y=FAKE + 2, ydt=2), dict(st=FAKE + 2)])
def test_matmul_refuses(L, kw):
    a = dict(xc=FAKE, xs=FAKE, fmt=0, wc=FAKE, ws=FAKE, M=4, N=8, K=64, y=FAKE, ydt=0, st=None)
    a.update(kw)
    assert L.qmoe_mx_matmul(a["xc"], a["xs"], a["fmt"], a["wc"], a["ws"], a["M"], a["N"], a["K"], a["y"], a["ydt"],
                            a["st"], None) == 1


def test_sizes_beyond_2_30_are_unsupported(L):
    big = (1 << 30) + 32
    for R, K in ((big, 64), (4, big)):
        assert L.qmoe_mx_quantize(FAKE, 0, 0, R, K, FAKE, FAKE, None) == 2
        assert L.qmoe_mx_dequant(FAKE, FAKE, 0, R, K, FAKE, 0, None) == 2
        assert L.qmoe_rmsnorm_mx(FAKE, None, None, 0, R, K, 0.0, 0, None, FAKE, FAKE, None) == 2
        assert L.qmoe_mx_matmul(FAKE, FAKE, 0, FAKE, FAKE, R, 8, K, FAKE, 0, None, None) == 2
    assert L.qmoe_mx_matmul(FAKE, FAKE, 0, FAKE, FAKE, 8, big, 64, FAKE, 0, None, None) == 2


@pytest.mark.parametrize("kw", [dict(i=None), dict(o=None), dict(R=0), dict(K=33)])
def test_scale_adapters_refuse(L, kw):
    a = dict(i=FAKE, o=FAKE, R=4, K=64)
    a.update(kw)
    for f in (L.qmoe_mx_tile_scales, L.qmoe_mx_untile_scales):
        assert f(a["i"], a["R"], a["K"], a["o"], None) == 1
    assert L.qmoe_mx_tile_scales(FAKE, 4, 64, FAKE + 8, None) == 1
    assert L.qmoe_mx_untile_scales(FAKE + 8, 4, 64, FAKE, None) == 1


def test_binding_refuses_what_it_cannot_pass_on(L):
    """Host tensors, wrong types, shapes and formats never reach the library."""
    from int4_block_quantized_gb300 import binding as B
    x, c, s = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    for call in (lambda: B.qmoe_mx_quantize(x), lambda: B.qmoe_mx_quantize(x, 5),
                 lambda: B.qmoe_mx_dequant(c, s, B.MXFP8), lambda: B.qmoe_mx_dequant(c, s, 2),
                 lambda: B.qmoe_rmsnorm_mx(x.half()), lambda: B.qmoe_mx_matmul(c, s, B.MXFP8, c, s),
                 lambda: B.qmoe_mx_tile_scales(c), lambda: B.qmoe_mx_untile_scales(s, 4, 64)):
        with pytest.raises(B.QMoEError) as e:
            call()
        assert e.value.code == 1


@pytest.mark.parametrize("R,K", [((1 << 30) + 1, 64), (2 ** 31 - 1, 32), (4, (1 << 30) + 32), (1, 2 ** 31 - 96),
                                 (129, 2 ** 31 - 32)])
def test_scale_adapters_beyond_2_30_are_unsupported(L, R, K):
    """Past the limit the kernels' 32-bit tile counts would overflow."""
    for f in (L.qmoe_mx_tile_scales, L.qmoe_mx_untile_scales):
        assert f(FAKE, R, K, FAKE, None) == 2


class Sized:
    """What the binding asks of a tensor before a call, at a size that no host holds."""

    def __init__(self, shape, dtype=torch.uint8):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda", 0)

    def numel(self):
        return self.shape.numel()

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return FAKE


def test_binding_refuses_sizes_that_the_abi_cannot_carry(L, monkeypatch):
    """A size beyond 32 bits would reach the library as another one (2^32 + 32
    columns as 32): it is refused before the call."""
    from int4_block_quantized_gb300 import binding as B
    calls = []
    monkeypatch.setattr(B, "_mx_call", lambda dev, fn, where, *args: calls.append(where))
    big, n = 2 ** 32 + 32, B.qmoe_mx_scale_bytes

    def mx_of(R, K, fmt):
        return Sized((R, K >> fmt)), Sized((n(R, K),))
    for R, K in ((1, big), (big, 64), (1, 2 ** 31), (2 ** 31, 32), (2 ** 30 + 1, 32), (1, 2 ** 30 + 32)):
        for fmt in (B.MXFP8, B.MXFP4):
            c, s = mx_of(R, K, fmt)
            small = mx_of(4, K, fmt)
            x = Sized((R, K), torch.float16)
            for call in (lambda: B.qmoe_mx_quantize(x, fmt, c, s),
                         lambda: B.qmoe_mx_dequant(c, s, fmt, torch.float16, x),
                         lambda: B.qmoe_rmsnorm_mx(x, fmt=fmt, codes=c, scales=s),
                         lambda: B.qmoe_mx_matmul(c, s, fmt, *mx_of(4, K, B.MXFP4), torch.float16, Sized((R, 4), torch.float16)),
                         lambda: B.qmoe_mx_matmul(*small, fmt, *mx_of(R, K, B.MXFP4), torch.float16, Sized((4, R), torch.float16))):
                with pytest.raises(B.QMoEError) as e:
                    call()
                assert e.value.code == 2
        for call in (lambda: B.qmoe_mx_tile_scales(Sized((R, K // 32))), lambda: B.qmoe_mx_untile_scales(Sized((n(R, K),)), R, K)):
            with pytest.raises(B.QMoEError) as e:
                call()
            assert e.value.code == 2
    assert not calls
    # the largest that passes reaches the library
    B.qmoe_mx_quantize(Sized((1, 2 ** 30), torch.float16), B.MXFP8, *mx_of(1, 2 ** 30, B.MXFP8))
    assert calls == ["qmoe_mx_quantize"]


def test_binding_refuses_shapes_that_only_count_right(L, monkeypatch):
    """As many elements in another shape would be read or written in another
    order than the caller's shape says."""
    from int4_block_quantized_gb300 import binding as B
    calls = []
    monkeypatch.setattr(B, "_mx_call", lambda dev, fn, where, *args: calls.append(where))
    f16, M, N, K = torch.float16, 4, 8, 64
    s, ws, wc = Sized((512,)), Sized((512,)), Sized((N, K // 2))
    x, c = Sized((M, K), f16), Sized((M, K))
    for shape in ((K, M), (M * K,), (2, M // 2, K), (M, K, 1)):
        t, u = Sized(shape, f16), Sized(shape)
        for call in (lambda: B.qmoe_mx_quantize(x, B.MXFP8, u, s), lambda: B.qmoe_mx_dequant(c, s, B.MXFP8, f16, t),
                     lambda: B.qmoe_rmsnorm_mx(x, t, codes=c, scales=s, residual_out=x),
                     lambda: B.qmoe_rmsnorm_mx(x, x, codes=c, scales=s, residual_out=t),
                     lambda: B.qmoe_rmsnorm_mx(x, codes=u, scales=s)):
            with pytest.raises(B.QMoEError) as e:
                call()
            assert e.value.code == 1
    for shape in ((N, M), (M * N,), (M // 2, 2 * N)):
        with pytest.raises(B.QMoEError) as e:
            B.qmoe_mx_matmul(c, s, B.MXFP8, wc, ws, f16, Sized(shape, f16))
        assert e.value.code == 1
    for shape in ((K, 1), (2, K // 2)):
        with pytest.raises(B.QMoEError) as e:
            B.qmoe_rmsnorm_mx(x, weight=Sized(shape, f16), codes=c, scales=s)
        assert e.value.code == 1
    assert not calls
    B.qmoe_mx_quantize(x, B.MXFP8, c, s)
    B.qmoe_mx_quantize(x, B.MXFP4, Sized((M, K // 2)), s)
    B.qmoe_mx_dequant(c, s, B.MXFP8, f16, x)
    for w in (None, Sized((K,), f16), Sized((1, K), f16)):  # a weight per column: broadcasting's shapes
        B.qmoe_rmsnorm_mx(x, x, w, codes=c, scales=s, residual_out=x)
    B.qmoe_mx_matmul(c, s, B.MXFP8, wc, ws, f16, Sized((M, N), f16))
    assert len(calls) == 7


def test_diagnosed_product_refuses_unknown_flags(L):
    for flags in (32, 63, 1 << 31):
        assert L.qmoe_mx_matmul_diagnosed(FAKE, FAKE, 0, FAKE, FAKE, 4, 8, 64, FAKE, 0, None, 1, flags, None) == 1
    assert L.qmoe_mx_matmul_diagnosed(FAKE, FAKE, 0, FAKE, FAKE, 4, 8, 65, FAKE, 0, None, 1, 1, None) == 1


def test_variant_query_refuses(L):
    import ctypes
    v = (ctypes.c_int * 4)()
    for a in ((2, FAKE, 4, 8, 64), (0, None, 4, 8, 64), (0, FAKE + 8, 4, 8, 64), (0, FAKE, 0, 8, 64), (0, FAKE, 4, 0, 64),
              (0, FAKE, 4, 8, 48)):
        assert L.qmoe_mx_matmul_variant(*a, v) == 1
    assert L.qmoe_mx_matmul_variant(0, FAKE, 4, 8, 64, None) == 1
    assert L.qmoe_mx_matmul_variant(0, FAKE, (1 << 30) + 1, 8, 64, v) == 2
