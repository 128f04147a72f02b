"""FP8 experts as measured work: quantisation with a scale for each block of 128, the product of such tensors (dense
or grouped by expert), tokens sorted by expert, and their weighted way back with its gradient.

An FP8 tensor is a tensor of e4m3 bytes and fp32 scales: activations [M, K] have one scale per row and 128 columns,
weights [E, N, K] one per 128 rows and 128 columns; the last block of a row or column may be shorter. With a the
largest magnitude of a block, at least 2^-100, its scale is fp32(a / 448), and a code is v * fp32(448 / a) rounded
to nearest even.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
LEAST = 2.0 ** -100


def listed():
    return [
        # one decoded token's hidden state to 8 bits: the latency of the smallest call
        {"name": "quantize 1 token", "op": "rows", "T": 1, "k": 0, "E": 0, "K": 2048, "x": "f16", "pad": 0},
        # a 2048-token stack layer: each token's state quantised in the order of the experts that it goes to
        {"name": "quantize sorted tokens", "op": "rows", "T": 2048, "k": 4, "E": 60, "K": 2048, "x": "bf16", "pad": 37},
        # the same layer between the experts' two products: SwiGLU of gate and up, to 8 bits
        {"name": "quantize swiglu", "op": "swiglu", "M": 8192, "K": 1408, "x": "bf16"},
        # loading a layer: the gate projections of 60 experts
        {"name": "quantize layer weights", "op": "weights", "E": 60, "N": 1408, "K": 2048, "x": "f16"},
        # one decoded token through gate and up of its four experts: the weights' bytes and the latency count
        {"name": "experts 1 token", "op": "product", "T": 1, "k": 4, "E": 60, "N": 2816, "K": 2048, "y": "f16", "pad": 0},
        # the 2048-token stack layer through gate and up: about 137 tokens an expert, unequal, some rows unused
        {"name": "experts 2048 tokens", "op": "product", "T": 2048, "k": 4, "E": 60, "N": 2816, "K": 2048, "y": "bf16", "pad": 37},
        # odd numbers of tokens and outputs, a ragged reduction, 32-bit result (logits)
        {"name": "product ragged", "op": "product", "T": 333, "k": 0, "E": 1, "N": 4099, "K": 1424, "y": "f32", "pad": 0},
        # a large square product: the tensor cores' rate counts
        {"name": "product 8192", "op": "product", "T": 8192, "k": 0, "E": 1, "N": 8192, "K": 8192, "y": "bf16", "pad": 0},
        # one decoded token handed to its experts: sort and gather, latency alone
        {"name": "dispatch 1 token", "op": "dispatch", "T": 1, "k": 4, "E": 60, "K": 2048, "x": "f16", "pad": 0},
        # a large prefill over many experts, its last tokens padding
        {"name": "dispatch 16384 tokens", "op": "dispatch", "T": 16384, "k": 8, "E": 256, "K": 2048, "x": "bf16", "pad": 301},
        # a speculative-verify batch's way back, onto the residual
        {"name": "combine 16 tokens", "op": "combine", "T": 16, "k": 4, "E": 60, "K": 2048, "x": "f16", "back": 0, "pad": 0},
        # the gradient of a large batch's way there and back: of the experts' outputs, the weights and the tokens
        {"name": "combine 16384 tokens back", "op": "combine", "T": 16384, "k": 8, "E": 128, "K": 2048, "x": "bf16", "back": 1, "pad": 301},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["rows", "swiglu", "weights", "product", "product", "product", "dispatch", "combine", "combine"])
    x, T, E = rng.choice(["bf16", "f16", "f32"]), _log(rng, 1, 8192), rng.choice([8, 60, 60, 128, 256])
    pad = rng.choice([0, T // 50])
    if op == "swiglu":
        return {"op": op, "M": T, "K": 16 * _log(rng, 1, 352), "x": x}
    if op == "weights":
        return {"op": op, "E": rng.choice([1, 8, 60]), "N": _log(rng, 8, 1408), "K": 16 * _log(rng, 8, 128), "x": x}
    if op == "rows":
        k = rng.choice([0, 1, 4, 8])
        return {"op": op, "T": T, "k": k, "E": E if k else 0, "K": 16 * _log(rng, 1, 128), "x": x, "pad": pad if k else 0}
    if op == "product" and rng.random() < 0.5:
        return {"op": op, "T": T, "k": 0, "E": 1, "N": _log(rng, 8, 8192), "K": 16 * _log(rng, 8, 512), "y": x, "pad": 0}
    if op == "product":
        T = _log(rng, 1, 2048)
        return {"op": op, "T": T, "k": rng.choice([1, 2, 4, 8]), "E": E, "N": _log(rng, 64, 1408), "K": 16 * _log(rng, 8, 128),
                "y": x, "pad": rng.choice([0, T // 50])}
    c = {"op": op, "T": T, "k": rng.choice([1, 2, 4, 8]), "E": E, "K": 8 * _log(rng, 8, 256), "x": x, "pad": pad}
    return {**c, "back": rng.choice([0, 1])} if op == "combine" else c


# ---- making inputs: seeded values, and codes, scales and orders put together apart from what is measured

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _hidden(g, rows, cols):
    """Hidden states: unit normal, rows of differing size, some channels that stand out."""
    v = torch.randn((rows, cols), generator=g, device=DEV)
    v *= torch.exp(0.5 * torch.randn((rows, 1), generator=g, device=DEV))
    v *= torch.where(torch.rand((1, cols), generator=g, device=DEV) < 0.01, 8.0, 1.0)
    return v


def _routing(g, T, k, E, pad):
    """(weights [T, k], ids [T, k]) of a router: softmax of logits that favour some experts, the k best of them. The
    last `pad` tokens are padding and go nowhere."""
    logits = 0.9 * torch.randn((T, E), generator=g, device=DEV) + 0.5 * torch.randn((1, E), generator=g, device=DEV)
    w, ids = torch.softmax(logits, -1).topk(k, -1)
    ids = ids.int()
    if pad:
        ids[T - pad:] = -1
    return w.contiguous(), ids.contiguous()


def _order(ids, E):
    """(offsets [E + 1], assignments by expert with -1 behind the last, place of each assignment or -1), int32."""
    flat = ids.flatten().long()
    flat = torch.where(flat < 0, E, flat)
    by, perm = torch.sort(flat, stable=True)
    pos = torch.empty_like(perm)
    pos[perm] = torch.arange(flat.numel(), device=ids.device)
    offsets = torch.searchsorted(by, torch.arange(E + 1, device=ids.device))
    return (offsets.int(), torch.where(by < E, perm, -1).int(), torch.where(flat < E, pos, -1).int().view(ids.shape))


def _codes(g, *shape):
    """e4m3 codes as a quantiser leaves them: magnitudes up to 448, most within six binades of it, and no NaN."""
    c = torch.randint(0, 2, shape, generator=g, device=DEV, dtype=torch.uint8) << 7
    return c | (126 - (torch.randn(shape, generator=g, device=DEV).abs_() * 20).to(torch.uint8).clamp_(max=126))


def _scales(g, *shape):
    return 0.01 * torch.exp(0.5 * torch.randn(shape, generator=g, device=DEV))


def _blocks(n):
    return -(-n // 128)


def prepare(case, seed):
    g, c = _gen(seed), case
    st, K = {"case": dict(c)}, c["K"]
    if c["op"] == "swiglu":
        st["h"] = _hidden(g, c["M"], 2 * K).to(DT[c["x"]])
        return st
    if c["op"] == "weights":
        st["w"] = (0.02 * torch.randn((c["E"], c["N"], K), generator=g, device=DEV)).to(DT[c["x"]])
        return st
    T, k, E = c["T"], c["k"], c["E"]
    rows = T * max(k, 1)
    if k:
        st["weights"], st["ids"] = _routing(g, T, k, E, c["pad"])
        st["offsets"], st["perm"], st["pos"] = _order(st["ids"], E)
    if c["op"] == "product":
        st["x_codes"], st["x_scales"] = _codes(g, rows, K), _scales(g, rows, _blocks(K))
        st["w_codes"], st["w_scales"] = _codes(g, E, c["N"], K), _scales(g, E, _blocks(c["N"]), _blocks(K))
        if k:
            st["most"] = int(torch.diff(st["offsets"]).max())  # tokens of the busiest expert: the plain form's padding
            st["out"] = torch.zeros((rows, c["N"]), dtype=DT[c["y"]], device=DEV)  # rows behind the last expert's stay
        return st
    if c["op"] == "combine":
        st["ys"] = _hidden(g, rows, K).to(DT[c["x"]])
        st["residual" if not c["back"] else "dout"] = _hidden(g, T, K).to(DT[c["x"]])
        if c["back"]:
            st["dxs"] = _hidden(g, rows, K).to(DT[c["x"]])
            st["dys"] = torch.zeros((rows, K), dtype=DT[c["x"]], device=DEV)
        return st
    st["x"] = _hidden(g, T, K).to(DT[c["x"]])
    if c["op"] == "rows" and k:
        st["codes"] = torch.zeros((rows, K), dtype=torch.uint8, device=DEV)
        st["scales"] = torch.zeros((rows, _blocks(K)), device=DEV)
    if c["op"] == "dispatch":
        st["xs"] = torch.zeros((rows, K), dtype=DT[c["x"]], device=DEV)
    return st


# ---- the plain forms

def _power(e):
    """2^e in 64 bits, from the bits (a power function may miss by the last one)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(a):
    """Nearest e4m3 magnitude, ties to even, at most 448 (64 bits, so that an exact product is rounded once)."""
    a = a.clamp(max=448.0)
    step = _power((torch.frexp(a)[1] - 1).clamp(min=-6) - 3)
    return torch.round(a / step) * step


def _pad(v, dim):
    """v with zeros behind it along dim, to whole blocks of 128."""
    n = -v.shape[dim] % 128
    if not n:
        return v
    shape = list(v.shape)
    shape[dim] = n
    return torch.cat((v, torch.zeros(shape, dtype=v.dtype, device=v.device)), dim)


def _plain_quantize(v, dim):
    """Values and scales of v's blocks, the dimensions `dim` of a view in which they lie whole. 32 bits but for the codes."""
    a = v.abs().amax(dim, keepdim=True).float().clamp(min=LEAST)
    top = torch.full_like(a, 448.0)  # a tensor: by a number, torch multiplies with a rounded reciprocal
    r, s = top / a, a / top
    q = torch.copysign(_e4m3((v.double() * r.double()).abs()), v.double())
    return (q * s.double()).float(), s


def _plain_rows(v):
    M, K = v.shape
    q, s = _plain_quantize(_pad(v, 1).view(M, -1, 128), 2)
    return q.view(M, -1)[:, :K], s[..., 0]


def _plain_weights(w):
    E, N, K = w.shape
    p = _pad(_pad(w, 1), 2)
    q, s = _plain_quantize(p.view(E, p.shape[1] // 128, 128, p.shape[2] // 128, 128), (2, 4))
    return q.reshape(p.shape)[:, :N, :K], s[:, :, 0, :, 0]


def _wide(scales, n, dim):
    return torch.repeat_interleave(scales, 128, dim).narrow(dim, 0, n)


def _plain_product(st, c):
    x = st["x_codes"].view(torch.float8_e4m3fn).float() * _wide(st["x_scales"], c["K"], 1)
    wc, ws = st["w_codes"], st["w_scales"]
    values = lambda codes, s: codes.view(torch.float8_e4m3fn).float() * _wide(_wide(s, c["N"], 1), c["K"], 2)  # noqa: E731
    if not c["k"]:
        return (x @ values(wc, ws)[0].t()).to(DT[c["y"]])
    offsets, rows = st["offsets"].long(), torch.arange(x.shape[0], device=x.device)
    used = (rows < offsets[-1])[:, None]
    expert = torch.searchsorted(offsets, rows, right=True).sub(1).clamp(max=c["E"] - 1)
    if x.shape[0] <= c["E"]:  # few rows: each with its own expert's weights
        y = torch.bmm(values(wc[expert], ws[expert]), x[:, :, None])[:, :, 0]
    else:  # every expert's rows, padded to those of the busiest
        at = (offsets[:-1, None] + torch.arange(st["most"], device=x.device)).clamp(max=x.shape[0] - 1)
        y = torch.bmm(x[at], values(wc, ws).transpose(1, 2))[expert, (rows - offsets[expert]).clamp(0, st["most"] - 1)]
    return torch.where(used, y, 0.0).to(DT[c["y"]])


def _gathered(x, perm, k):
    """Row perm / k of x for each place, zeros where there is none."""
    return torch.where(perm[:, None] >= 0, x[(perm.clamp(min=0) // k).long()], torch.zeros_like(x[:1]))


def run(state):
    c, st = state["case"], state
    if own:
        from int4_block_quantized_gb300 import binding as B
        if c["op"] == "rows":
            if c["k"]:
                codes, scales = B.qmoe_fp8_quantize(st["x"], st["pos"], codes=st["codes"], scales=st["scales"])
            else:
                codes, scales = B.qmoe_fp8_quantize(st["x"])
            return {"scales": scales, "values": B.qmoe_fp8_dequant(codes, scales, torch.bfloat16)}
        if c["op"] == "swiglu":
            codes, scales = B.qmoe_fp8_quantize_swiglu(st["h"])
            return {"scales": scales, "values": B.qmoe_fp8_dequant(codes, scales, torch.bfloat16)}
        if c["op"] == "weights":
            codes, scales = B.qmoe_fp8_quantize_weights(st["w"])
            return {"scales": scales, "values": B.qmoe_fp8_dequant(codes, scales, torch.bfloat16)}
        if c["op"] == "product":
            return {"y": B.qmoe_fp8_matmul(st["x_codes"], st["x_scales"], st["w_codes"], st["w_scales"], DT[c["y"]],
                                           offsets=st.get("offsets"), out=st.get("out"))}
        if c["op"] == "dispatch":
            offsets, perm, pos = B.qmoe_sort_experts(st["ids"], c["E"])
            return {"offsets": offsets, "perm": perm, "pos": pos, "xs": B.qmoe_dispatch(st["x"], pos, out=st["xs"])}
        if not c["back"]:
            return {"out": B.qmoe_combine(st["ys"], st["pos"], st["weights"], st["residual"])}
        dys, dw = B.qmoe_combine_backward(st["dout"], st["ys"], st["pos"], st["weights"], dys=st["dys"])
        return {"dys": dys, "dw": dw, "dx": B.qmoe_dispatch_backward(st["dxs"], st["pos"])}
    if c["op"] == "rows":
        x = st["x"].float()
        if not c["k"]:
            q, s = _plain_rows(x)
        else:
            q, s = _plain_rows(_gathered(x, st["perm"], c["k"]))
            s = torch.where(st["perm"][:, None] >= 0, s, 0.0)
        return {"scales": s, "values": q.to(torch.bfloat16)}
    if c["op"] == "swiglu":
        g, u = st["h"].double().split(c["K"], 1)  # 64 bits: values next to a border between two codes
        q, s = _plain_rows(g / (1 + torch.exp(-g)) * u)
        return {"scales": s, "values": q.to(torch.bfloat16)}
    if c["op"] == "weights":
        q, s = _plain_weights(st["w"].float())
        return {"scales": s, "values": q.to(torch.bfloat16)}
    if c["op"] == "product":
        return {"y": _plain_product(st, c)}
    if c["op"] == "dispatch":
        offsets, perm, pos = _order(st["ids"], c["E"])
        return {"offsets": offsets, "perm": perm, "pos": pos, "xs": _gathered(st["x"], perm, c["k"])}
    pos, dt = st["pos"], DT[c["x"]]
    there, at = (pos >= 0)[..., None], pos.clamp(min=0).long()
    ys = torch.where(there, st["ys"][at].float(), 0.0)  # [T, k, H]
    if not c["back"]:
        return {"out": (st["residual"].float() + (st["weights"][..., None] * ys).sum(1)).to(dt)}
    dout = st["dout"].float()[:, None]
    dw = (dout * ys).sum(-1)
    perm = st["perm"]
    t, j = (perm.clamp(min=0) // c["k"]).long(), (perm.clamp(min=0) % c["k"]).long()
    dys = torch.where(perm[:, None] >= 0, st["weights"][t, j][:, None] * st["dout"].float()[t], 0.0)
    dx = torch.where(there, st["dxs"][at].float(), 0.0).sum(1)
    return {"dys": dys.to(dt), "dw": dw, "dx": dx.to(dt)}


def work(case):
    c, K = case, case["K"]
    q = 1 + 4 / 128  # bytes of an element with its share of a row's scale
    if c["op"] == "swiglu":  # gate and up in; codes and scales out and in again, values out
        n = c["M"] * K
        return {"bytes": n * (2 * SIZE[c["x"]] + 2 * q + 2), "flops": 12 * n}
    if c["op"] == "weights":
        n = c["E"] * c["N"] * K
        return {"bytes": n * (SIZE[c["x"]] + 2 + 2), "flops": 4 * n}
    T, k, E = c["T"], c["k"], c["E"]
    used = (T - c["pad"]) * max(k, 1)
    if c["op"] == "rows":
        return {"bytes": (T - c["pad"]) * K * SIZE[c["x"]] + used * (K * (2 * q + 2) + (4 if k else 0)), "flops": 4 * used * K}
    if c["op"] == "product":
        N, experts = c["N"], min(E, used)
        return {"bytes": used * K * q + experts * N * K + used * N * SIZE[c["y"]], "flops": 2 * used * N * K}
    size = K * SIZE[c["x"]]
    if c["op"] == "dispatch":
        return {"bytes": (T - c["pad"]) * size + used * size + 12 * T * k + 4 * E, "flops": 4 * T * k}
    if not c["back"]:
        return {"bytes": used * size + 2 * T * size + 8 * T * k, "flops": 2 * used * K}
    return {"bytes": 3 * used * size + 2 * T * size + 16 * T * k, "flops": 4 * used * K}


# ---- the definitions in 64 bits, from the list of values that the format has

def _nearest(a):
    """Nearest e4m3 magnitude of a >= 0, an exact middle to the one with the even code."""
    grid = torch.tensor([m / 512 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1],
                        dtype=torch.float64, device=a.device)
    middle = (grid[1:] + grid[:-1]) / 2
    below, above = torch.bucketize(a, middle), torch.bucketize(a, middle, right=True)
    return grid[torch.where((below != above) & (below % 2 == 1), above, below)]


def _exact_block(v):
    """v [n, b] in 64 bits, each row a block -> values, scales [n]."""
    big = v.abs().max(1).values.clamp(min=LEAST)
    s = (big / 448).float().double()
    q = _nearest(v.abs() * (448 / big.float().double()).float().double()[:, None])
    return q * torch.sign(v) * s[:, None], s


def _exact_rows(v):
    M, K = v.shape
    out, s = torch.zeros_like(v), torch.zeros((M, _blocks(K)), dtype=torch.float64, device=v.device)
    for b in range(_blocks(K)):
        out[:, 128 * b:128 * b + 128], s[:, b] = _exact_block(v[:, 128 * b:128 * b + 128])
    return out, s


def _exact_values(codes):
    c = codes.long()
    e, m = c >> 3 & 15, (c & 7).double()
    mag = torch.where(e == 0, m / 512, (1 + m / 8) * _power(e - 7))
    return torch.where(c >> 7 == 1, -mag, mag)


def exact(case, seed):
    st, c, K = prepare(case, seed), case, case["K"]
    if c["op"] == "swiglu":
        g, u = st["h"][:, :K].double(), st["h"][:, K:].double()
        v, s = _exact_rows(g * torch.sigmoid(g) * u)
        return {"scales": s, "values": v}
    if c["op"] == "weights":
        E, N = c["E"], c["N"]
        v = torch.empty((E, N, K), dtype=torch.float64, device=DEV)
        s = torch.empty((E, _blocks(N), _blocks(K)), dtype=torch.float64, device=DEV)
        for n in range(_blocks(N)):
            for b in range(_blocks(K)):
                part = st["w"][:, 128 * n:128 * n + 128, 128 * b:128 * b + 128].double()
                q, s[:, n, b] = _exact_block(part.reshape(E, -1))
                v[:, 128 * n:128 * n + 128, 128 * b:128 * b + 128] = q.view(part.shape)
        return {"scales": s, "values": v}
    T, k = c["T"], c["k"]
    used = int(st["offsets"][-1]) if k else T
    token = st["perm"][:used].long() // k if k else None
    if c["op"] == "rows":
        v, s = _exact_rows(st["x"].double() if not k else st["x"].double()[token])
        if k:
            v = torch.cat((v, torch.zeros((T * k - used, K), dtype=v.dtype, device=DEV)))
            s = torch.cat((s, torch.zeros((T * k - used, s.shape[1]), dtype=s.dtype, device=DEV)))
        return {"scales": s, "values": v}
    if c["op"] == "product":
        each = torch.arange(K, device=DEV) // 128
        x = _exact_values(st["x_codes"]) * st["x_scales"].double()[:, each]
        y = torch.zeros((x.shape[0], c["N"]), dtype=torch.float64, device=DEV)
        ends = st["offsets"].tolist() if k else [0, T]
        for e in range(c["E"]):
            a, b = ends[e], ends[e + 1]
            if a < b:
                w = _exact_values(st["w_codes"][e]) * st["w_scales"][e].double()[torch.arange(c["N"], device=DEV) // 128][:, each]
                y[a:b] = torch.einsum("mk,nk->mn", x[a:b], w)
        return {"y": y}
    if c["op"] == "dispatch":
        xs = torch.zeros((T * k, K), dtype=torch.float64, device=DEV)
        xs[:used] = st["x"].double()[token]
        return {"offsets": None, "perm": None, "pos": None, "xs": xs}
    ys, w = st["ys"].double(), st["weights"].double()
    choice = st["perm"][:used].long() % k
    if not c["back"]:
        out = st["residual"].double().clone()
        out.index_add_(0, token, w[token, choice][:, None] * ys[:used])
        return {"out": out}
    dout = st["dout"].double()
    dys = torch.zeros_like(ys)
    dys[:used] = w[token, choice][:, None] * dout[token]
    dw = torch.zeros_like(w)
    dw[token, choice] = (ys[:used] * dout[token]).sum(1)
    dx = torch.zeros_like(dout)
    dx.index_add_(0, token, st["dxs"][:used].double())
    return {"dys": dys, "dw": dw, "dx": dx}
