"""The FP8 experts' calls with some of their outputs left out: what is left is bit for
bit what the full calls give, and nothing else is written."""
import pytest
import torch

from int4_block_quantized_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32, I32 = torch.float16, torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int4_block_quantized_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def ids_of(T, k, E, drop=0.2):
    g = torch.Generator().manual_seed(T + k + E)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=I32)
    ids[torch.rand((T, k), generator=g) < drop] = -1
    return ids.to(DEV)


# one CTA, one cluster of 8, one of 16; both numbers of votes
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 4, 60), (300, 2, 256), (3000, 2, 8), (3000, 2, 128), (10000, 4, 60), (9000, 4, 256)])
def test_sort_without_some_outputs(T, k, E):
    ids = ids_of(T, k, E)
    full = B.qmoe_sort_experts(ids, E)
    names = ("offsets", "perm", "pos")
    for wanted in range(8):
        bufs = [torch.full((3,) + t.shape, 99, dtype=I32, device=DEV) for t in full]
        out = B.qmoe_sort_experts(ids, E, **{n: bufs[i][1] if wanted >> i & 1 else False for i, n in enumerate(names)})
        for i in range(3):
            if wanted >> i & 1:
                assert torch.equal(out[i], full[i]) and torch.equal(bufs[i][1], full[i]) and (bufs[i][::2] == 99).all()
            else:
                assert out[i] is None and (bufs[i] == 99).all()


@pytest.mark.parametrize("ydt,odt", [(F16, F16), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("T,k,E,H", [(1, 4, 60, 2048), (3, 1, 2, 8), (40, 3, 5, 24), (200, 8, 60, 1000), (65, 2, 7, 2056)])
def test_combine_backward_without_one_gradient(T, k, E, H, ydt, odt):
    g = torch.Generator(device=DEV).manual_seed(T)
    pos = B.qmoe_sort_experts(ids_of(T, k, E), E)[2]
    dout, ys = torch.randn((T, H), generator=g, device=DEV).to(odt), torch.randn((T * k, H), generator=g, device=DEV).to(ydt)
    for w in (torch.rand((T, k), generator=g, device=DEV), None):
        mark = lambda: torch.full((T * k, H), 7.0, dtype=ydt, device=DEV)  # noqa: E731
        dys, dw = B.qmoe_combine_backward(dout, ys, pos, w, dys=mark())
        for y in (ys, None):
            only, none = B.qmoe_combine_backward(dout, y, pos, w, dys=mark(), dw=False)
            assert none is None and torch.equal(only, dys)
        before = ys.clone()
        none, only = B.qmoe_combine_backward(dout, ys, pos, w, dys=False)
        assert none is None and torch.equal(only, dw) and torch.equal(ys, before)
        only, none = B.qmoe_combine_backward(dout, ys, pos, w, dys=ys.clone(), dw=False)
        there = torch.zeros(T * k, dtype=torch.bool, device=DEV)
        there[pos[pos >= 0].long()] = True
        assert torch.equal(only[there], dys[there]) and torch.equal(only[~there], ys[~there])


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("T,k,E,H", [(1, 4, 60, 2048), (3, 1, 2, 8), (70, 8, 60, 1000)])
def test_dispatch_backward_of_the_library(T, k, E, H, dtype):
    """The C entry, which the binding reaches through the combine, gives the same."""
    g = torch.Generator(device=DEV).manual_seed(T)
    pos = B.qmoe_sort_experts(ids_of(T, k, E), E)[2]
    dxs = torch.randn((T * k, H), generator=g, device=DEV).to(dtype)
    buf = torch.full((3, T, H), 7.0, dtype=dtype, device=DEV)
    rc = B.lib().qmoe_dispatch_backward(dxs.data_ptr(), B._MX_DT[dtype], pos.data_ptr(), T, H, k, buf[1].data_ptr(),
                                        torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and torch.equal(buf[1], B.qmoe_dispatch_backward(dxs, pos)) and (buf[::2] == 7).all()
