"""Outputs of the FP8 experts' calls that are not wanted, on the host (no GPU): what
reaches the library, and what the binding refuses."""
import pytest
import torch

FAKE = 0x10000  # 16-byte aligned, never dereferenced
F16, BF16, F32, I32 = torch.float16, torch.bfloat16, torch.float32, torch.int32


class Sized:
    """What the binding asks of a tensor before a call."""

    def __init__(self, shape, dtype, dev=0, contiguous=True, at=FAKE):
        self.shape, self.dtype, self.device, self.dev, self.c, self.at = torch.Size(shape), dtype, torch.device("cuda", max(dev, 0)), dev, contiguous, at

    def numel(self):
        return self.shape.numel()

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return self.c

    def data_ptr(self):
        return self.at


@pytest.fixture
def calls(monkeypatch):
    from int4_block_quantized_gb300 import binding as B, build
    build.build()
    B.lib()
    seen = []
    monkeypatch.setattr(B, "_mx_call", lambda dev, fn, where, *args: seen.append(args))
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=None, device=None: Sized(shape, dtype, at=FAKE + 0x1000))
    return seen


def test_sort_passes_null_for_what_is_not_wanted(calls):
    from int4_block_quantized_gb300 import binding as B
    ids, given = Sized((4, 2), I32), Sized((4, 2), I32, at=FAKE + 64)
    new = FAKE + 0x1000
    for kw, want in (({}, (new, new, new)), (dict(perm=False), (new, None, new)), (dict(offsets=False, perm=False, pos=given), (None, None, FAKE + 64)),
                     (dict(offsets=False, perm=False, pos=False), (None, None, None))):
        out = B.qmoe_sort_experts(ids, 8, **kw)
        assert calls.pop() == (FAKE, 4, 2, 8) + want
        assert [t is None for t in out] == [p is None for p in want]
    assert B.qmoe_sort_experts(ids, 8, pos=given)[2] is given


@pytest.mark.parametrize("name,shape", [("offsets", (9,)), ("perm", (8,)), ("pos", (4, 2))])
def test_sort_refuses_outputs_that_do_not_fit(calls, name, shape):
    from int4_block_quantized_gb300 import binding as B
    for bad in (Sized(shape, torch.int64), Sized(shape, I32, 1), Sized(shape, I32, -1), Sized(shape, I32, 0, False), Sized((shape[0] + 1,) + shape[1:], I32)):
        with pytest.raises(B.QMoEError) as e:
            B.qmoe_sort_experts(Sized((4, 2), I32), 8, **{name: bad})
        assert e.value.code == 1
    assert not calls


def test_combine_backward_passes_null_for_what_is_not_wanted(calls):
    from int4_block_quantized_gb300 import binding as B
    dout, ys, pos = Sized((4, 64), F32), Sized((8, 64), F16), Sized((4, 2), I32)
    new = FAKE + 0x1000
    dys, dw = B.qmoe_combine_backward(dout, ys, pos, dys=False)
    assert calls.pop() == (FAKE, 2, FAKE, 0, FAKE, None, 4, 64, 2, None, new) and dys is None and dw.shape == (4, 2)
    dys, dw = B.qmoe_combine_backward(dout, ys, pos, dw=False)
    assert calls.pop() == (FAKE, 2, FAKE, 0, FAKE, None, 4, 64, 2, new, None) and dw is None and dys.dtype is F16
    dys, dw = B.qmoe_combine_backward(dout, None, pos, dw=False)
    assert calls.pop() == (FAKE, 2, None, 2, FAKE, None, 4, 64, 2, new, None) and dys.dtype is F32 and dys.shape == (8, 64)
    given = Sized((8, 64), BF16)
    assert B.qmoe_combine_backward(dout, None, pos, dys=given, dw=False)[0] is given
    assert calls.pop() == (FAKE, 2, None, 1, FAKE, None, 4, 64, 2, FAKE, None)


def test_combine_backward_refuses(calls):
    from int4_block_quantized_gb300 import binding as B
    dout, ys, pos = Sized((4, 64), F32), Sized((8, 64), F16), Sized((4, 2), I32)
    for a, kw in (((dout, ys, pos), dict(dys=False, dw=False)), ((dout, None, pos), {}), ((dout, None, pos), dict(dys=False)),
                  ((dout, None, pos), dict(dys=Sized((8, 64), I32), dw=False)), ((dout, None, pos), dict(dys=Sized((4, 64), F16), dw=False)),
                  ((dout, None, pos), dict(dys=Sized((8, 64), F16, 1), dw=False)), ((dout, ys, pos), dict(dys=Sized((8, 64), F32), dw=False))):
        with pytest.raises(B.QMoEError) as e:
            B.qmoe_combine_backward(*a, **kw)
        assert e.value.code == 1
    assert not calls
