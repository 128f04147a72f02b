"""Host-side checks of the FP8 entry points (no GPU): bad arguments refused with
the documented status before anything is enqueued."""
import pytest
import torch

FAKE = 0x10000  # 16-byte aligned, never dereferenced: every call below fails its checks first
BIG = (1 << 30) + 16


@pytest.fixture(scope="module")
def L():
    from int4_block_quantized_gb300 import build as b
    b.build()
    from int4_block_quantized_gb300 import binding
    return binding.lib()


def call(f, defaults, kw):
    a = dict(defaults)
    assert set(kw) <= set(a)
    a.update(kw)
    return f(*a.values(), None)


QUANTIZE = dict(x=FAKE, xdt=0, T=4, K=64, pos=FAKE, k=2, c=FAKE, s=FAKE)
SWIGLU = dict(h=FAKE, hdt=1, M=4, I=48, c=FAKE, s=FAKE)
WEIGHTS = dict(w=FAKE, wdt=2, E=2, N=5, K=64, c=FAKE, s=FAKE)
DEQUANT = dict(c=FAKE, s=FAKE, E=2, N=5, K=64, rows=128, o=FAKE, odt=0)
MATMUL = dict(xc=FAKE, xs=FAKE, wc=FAKE, ws=FAKE, off=FAKE, E=2, M=4, N=8, K=64, y=FAKE, ydt=0, st=None)
SORT = dict(ids=FAKE, T=4, k=2, E=8, off=FAKE, perm=FAKE, pos=FAKE)
DISPATCH = dict(x=FAKE, dt=0, T=4, H=64, k=2, pos=FAKE, xs=FAKE)
DISPATCH_BACK = dict(d=FAKE, dt=0, pos=FAKE, T=4, H=64, k=2, dx=FAKE)
COMBINE = dict(ys=FAKE, ydt=0, pos=FAKE, w=FAKE, r=FAKE, T=4, H=64, k=2, o=FAKE, odt=0)
BACKWARD = dict(d=FAKE, ddt=0, ys=FAKE, ydt=0, pos=FAKE, w=FAKE, T=4, H=64, k=2, dys=FAKE, dw=FAKE)

INVALID = [
    ("qmoe_fp8_quantize", QUANTIZE, [dict(x=None), dict(x=FAKE + 8), dict(xdt=3), dict(xdt=-1), dict(T=0), dict(K=0), dict(K=8),
                                     dict(K=72), dict(pos=FAKE + 2), dict(k=0), dict(k=-1), dict(pos=None), dict(c=None),
                                     dict(c=FAKE + 8), dict(s=None), dict(s=FAKE + 2)]),
    ("qmoe_fp8_quantize_swiglu", SWIGLU, [dict(h=None), dict(h=FAKE + 8), dict(hdt=3), dict(M=0), dict(I=0), dict(I=40),
                                          dict(c=None), dict(c=FAKE + 4), dict(s=None), dict(s=FAKE + 1)]),
    ("qmoe_fp8_quantize_weights", WEIGHTS, [dict(w=None), dict(w=FAKE + 8), dict(wdt=4), dict(E=0), dict(N=0), dict(K=24),
                                            dict(c=None), dict(c=FAKE + 8), dict(s=None), dict(s=FAKE + 2)]),
    ("qmoe_fp8_dequant", DEQUANT, [dict(c=None), dict(c=FAKE + 8), dict(s=None), dict(s=FAKE + 2), dict(E=0), dict(N=0), dict(K=8),
                                   dict(rows=0), dict(rows=64), dict(o=None), dict(o=FAKE + 8), dict(odt=3)]),
    ("qmoe_fp8_matmul", MATMUL, [dict(xc=None), dict(xs=None), dict(wc=None), dict(ws=None), dict(xc=FAKE + 8),
                                 dict(xs=FAKE + 2), dict(wc=FAKE + 8), dict(ws=FAKE + 2), dict(off=FAKE + 2), dict(off=None),
                                 dict(E=0), dict(M=0), dict(N=0), dict(K=0), dict(K=40), dict(y=None), dict(y=FAKE + 1),
                                 dict(y=FAKE + 2, ydt=2), dict(ydt=3), dict(st=FAKE + 2)]),
    ("qmoe_sort_experts", SORT, [dict(ids=None), dict(ids=FAKE + 2), dict(T=0), dict(k=0), dict(E=0), dict(off=FAKE + 1),
                                 dict(perm=FAKE + 2), dict(pos=FAKE + 2)]),
    ("qmoe_dispatch", DISPATCH, [dict(x=None), dict(x=FAKE + 8), dict(dt=3), dict(T=0), dict(H=0), dict(H=12), dict(k=0),
                                 dict(pos=None), dict(pos=FAKE + 2), dict(xs=None), dict(xs=FAKE + 8)]),
    ("qmoe_dispatch_backward", DISPATCH_BACK, [dict(d=None), dict(d=FAKE + 8), dict(dt=3), dict(pos=None), dict(T=0), dict(H=4),
                                               dict(k=0), dict(dx=None), dict(dx=FAKE + 8)]),
    ("qmoe_combine", COMBINE, [dict(ys=None), dict(ys=FAKE + 8), dict(ydt=3), dict(pos=None), dict(pos=FAKE + 1), dict(w=FAKE + 2),
                               dict(r=FAKE + 8), dict(T=0), dict(H=20), dict(k=0), dict(o=None), dict(o=FAKE + 4), dict(odt=-1)]),
    ("qmoe_combine_backward", BACKWARD, [dict(d=None), dict(d=FAKE + 8), dict(ddt=3), dict(ys=None), dict(ys=FAKE + 8),
                                         dict(ydt=3), dict(pos=None), dict(w=FAKE + 2), dict(T=0), dict(H=20), dict(k=0),
                                         dict(dys=FAKE + 8), dict(dw=FAKE + 2), dict(dys=None, dw=None)]),
]


@pytest.mark.parametrize("name,defaults,kws", INVALID, ids=[i[0] for i in INVALID])
def test_invalid_arguments(L, name, defaults, kws):
    for kw in kws:
        assert call(getattr(L, name), defaults, kw) == 1, kw


@pytest.mark.parametrize("name,defaults,kws", [
    ("qmoe_fp8_quantize", QUANTIZE, [dict(T=BIG), dict(K=BIG), dict(T=1 << 20, k=1 << 11)]),
    ("qmoe_fp8_quantize_swiglu", SWIGLU, [dict(M=BIG), dict(I=BIG)]),
    ("qmoe_fp8_quantize_weights", WEIGHTS, [dict(N=BIG), dict(E=1 << 20, N=1 << 11), dict(K=BIG)]),
    ("qmoe_fp8_dequant", DEQUANT, [dict(N=BIG), dict(E=1 << 20, N=1 << 11), dict(K=BIG)]),
    ("qmoe_fp8_matmul", MATMUL, [dict(M=BIG), dict(N=BIG), dict(K=BIG), dict(E=257)]),
    ("qmoe_sort_experts", SORT, [dict(E=257), dict(T=1 << 30), dict(T=1 << 20, k=1 << 11)]),
    ("qmoe_dispatch", DISPATCH, [dict(T=1 << 30), dict(H=(1 << 28) + 8)]),
    ("qmoe_combine", COMBINE, [dict(T=1 << 30), dict(H=(1 << 28) + 8)]),
    ("qmoe_combine_backward", BACKWARD, [dict(T=1 << 30), dict(H=(1 << 28) + 8)]),
])
def test_sizes_beyond_the_limits_are_unsupported(L, name, defaults, kws):
    for kw in kws:
        assert call(getattr(L, name), defaults, kw) == 2, kw


class Sized:
    """What the binding asks of a tensor before a call, at a size that no host holds."""

    def __init__(self, shape, dtype=torch.uint8, dev=0, contiguous=True):
        self.shape, self.dtype, self.device, self.dev, self.c = torch.Size(shape), dtype, torch.device("cuda", max(dev, 0)), dev, contiguous

    def numel(self):
        return self.shape.numel()

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return self.c

    def data_ptr(self):
        return FAKE


@pytest.fixture
def calls(monkeypatch, L):
    from int4_block_quantized_gb300 import binding as B
    seen = []
    monkeypatch.setattr(B, "_mx_call", lambda dev, fn, where, *args: seen.append(where))
    return seen


F16, F32, I32, U8 = torch.float16, torch.float32, torch.int32, torch.uint8
# name -> (keyword arguments that pass, of tensors [shape, dtype])
GOOD = {
    "qmoe_fp8_quantize": dict(x=((4, 144), F16), pos=((4, 2), I32), codes=((8, 144), U8), scales=((8, 2), F32)),
    "qmoe_fp8_quantize_swiglu": dict(h=((4, 288), F32), codes=((4, 144), U8), scales=((4, 2), F32)),
    "qmoe_fp8_quantize_weights": dict(w=((3, 130, 144), F16), codes=((3, 130, 144), U8), scales=((3, 2, 2), F32)),
    "qmoe_fp8_dequant": dict(codes=((3, 130, 144), U8), scales=((3, 2, 2), F32), out=((3, 130, 144), torch.bfloat16)),
    "qmoe_fp8_matmul": dict(x_codes=((8, 144), U8), x_scales=((8, 2), F32), w_codes=((3, 130, 144), U8), w_scales=((3, 2, 2), F32),
                            offsets=((4,), I32), out=((8, 130), torch.bfloat16), status=((1,), I32)),
    "qmoe_dispatch": dict(x=((4, 64), F16), pos=((4, 2), I32), out=((8, 64), F16)),
    "qmoe_dispatch_backward": dict(dxs=((8, 64), F16), pos=((4, 2), I32), out=((4, 64), F16)),
    "qmoe_combine": dict(ys=((8, 64), F16), pos=((4, 2), I32), w=((4, 2), F32), residual=((4, 64), F32), out=((4, 64), F32)),
    "qmoe_combine_backward": dict(dout=((4, 64), F32), ys=((8, 64), F16), pos=((4, 2), I32), w=((4, 2), F32), dys=((8, 64), F16),
                                  dw=((4, 2), F32)),
}


@pytest.mark.parametrize("name", GOOD)
def test_binding_refuses_tensors_that_do_not_fit(calls, name):
    """Each tensor in turn: of another shape with as many elements, another type,
    not contiguous, on the host; nothing of it reaches the library."""
    from int4_block_quantized_gb300 import binding as B
    good = GOOD[name]
    getattr(B, name)(**{k: Sized(*v) for k, v in good.items()})
    assert calls == [name]
    for key, (shape, dtype) in good.items():
        n = torch.Size(shape).numel()
        bad = [Sized((n,) if len(shape) > 1 else (n, 1, 1), dtype), Sized(shape, torch.int64), Sized(shape, dtype, -1),
               Sized(shape, dtype, 0, False), Sized(shape, dtype, 1)]
        if len(shape) > 1:
            bad += [Sized(shape[::-1], dtype), Sized((shape[0] + 1,) + shape[1:], dtype)]
        if key == "status":
            bad = bad[1:]
        for t in bad:
            with pytest.raises(B.QMoEError) as e:
                getattr(B, name)(**{k: t if k == key else Sized(*v) for k, v in good.items()})
            assert e.value.code == 1, (key, t.shape, t.dtype)
    assert calls == [name]


def test_binding_refuses_ids(calls):
    from int4_block_quantized_gb300 import binding as B
    for ids, E, code in ((Sized((4, 2), torch.int64), 8, 1), (Sized((8,), I32), 8, 1), (Sized((0, 2), I32), 8, 1), (Sized((4, 2), I32), 0, 1),
                         (Sized((4, 2), I32), 257, 2), (Sized((1 << 29, 4), I32), 8, 2), (Sized((4, 2), I32, -1), 8, 1)):
        with pytest.raises(B.QMoEError) as e:
            B.qmoe_sort_experts(ids, E)
        assert e.value.code == code
    assert not calls


def test_binding_refuses_sizes_that_the_abi_cannot_carry(calls):
    from int4_block_quantized_gb300 import binding as B
    big = 2 ** 32 + 32
    for call in (lambda: B.qmoe_fp8_quantize(Sized((1, big), F16)), lambda: B.qmoe_fp8_quantize(Sized((big, 16), F16)),
                 lambda: B.qmoe_fp8_quantize(Sized((2 ** 28, 16), F16), Sized((2 ** 28, 16), I32)),
                 lambda: B.qmoe_fp8_quantize_swiglu(Sized((1, 2 * big), F16)), lambda: B.qmoe_fp8_quantize_weights(Sized((2 ** 16, 2 ** 16, 32), F16)),
                 lambda: B.qmoe_fp8_dequant(Sized((1, big)), Sized((1, (big + 127) // 128), F32)),
                 lambda: B.qmoe_fp8_matmul(Sized((big, 32)), Sized((big, 1), F32), Sized((8, 32)), Sized((1, 1), F32)),
                 lambda: B.qmoe_fp8_matmul(Sized((8, 32)), Sized((8, 1), F32), Sized((big, 32)), Sized((big // 128, 1), F32)),
                 lambda: B.qmoe_dispatch(Sized((2, big), F16), Sized((2, 2), I32)),
                 lambda: B.qmoe_combine(Sized((4, big), F16), Sized((2, 2), I32)),
                 lambda: B.qmoe_combine(Sized((2 ** 34, 8), F16), Sized((2 ** 32, 4), I32))):
        with pytest.raises(B.QMoEError) as e:
            call()
        assert e.value.code == 2
    assert not calls


def test_diagnosed_product_refuses_unknown_flags(L):
    a = [v for k, v in MATMUL.items()]
    for flags in (16, 31, 1 << 31):
        assert L.qmoe_fp8_matmul_diagnosed(*a, 1, flags, None) == 1
    assert call(L.qmoe_fp8_matmul, MATMUL, dict(K=40)) == 1


def test_variant_query_refuses(L):
    import ctypes
    v = (ctypes.c_int * 3)()
    for a in ((0, 2, 4, 8, 64), (1, 0, 4, 8, 64), (1, 2, 0, 8, 64), (1, 2, 4, 0, 64), (1, 2, 4, 8, 40)):
        assert L.qmoe_fp8_matmul_variant(*a, v) == 1
    assert L.qmoe_fp8_matmul_variant(1, 2, 4, 8, 64, None) == 1
    assert L.qmoe_fp8_matmul_variant(1, 257, 4, 8, 64, v) == 2 and L.qmoe_fp8_matmul_variant(0, 1, BIG, 8, 64, v) == 2
