"""The microscaled (MX) operators as measured work: quantisation and its reading back, the residual RMSNorm
with microscaled output, and the product with MXFP4 weights.

An MX tensor [R, K] is a tensor of codes (MXFP8: one e4m3 byte per element; MXFP4: two e2m1 codes per byte, even
k in the low nibble) and one e8m0 scale byte per block of 32 elements of a row, kept in tiles of 128 rows x 4
blocks: byte (r % 32) * 16 + (r % 128 / 32) * 4 + b % 4 of tile (r / 128, b / 4), tiles row-major, padding 0.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
EMAX = {"mxfp8": 8, "mxfp4": 2}
EPS = 1e-6


def listed():
    return [
        # one decoded token's hidden state to 8 bits: the latency of the smallest call
        {"name": "quantize 1 token", "op": "quantize", "M": 1, "K": 2048, "x": "bf16", "fmt": "mxfp8"},
        # a 2048-token prefill batch of the shared expert's intermediate state to 4 bits
        {"name": "quantize 2048 tokens", "op": "quantize", "M": 2048, "K": 5632, "x": "bf16", "fmt": "mxfp4"},
        # loading a layer: the gate projections of 60 experts (1408 x 2048 each) to MXFP4
        {"name": "quantize layer weights", "op": "quantize", "M": 84480, "K": 2048, "x": "f16", "fmt": "mxfp4"},
        # the norm in front of a layer, one decoded token
        {"name": "norm 1 token", "op": "norm", "M": 1, "K": 2048, "x": "f16", "fmt": "mxfp8"},
        # the same for a prefill batch with a ragged number of tokens
        {"name": "norm 509 tokens", "op": "norm", "M": 509, "K": 2048, "x": "bf16", "fmt": "mxfp8"},
        # a large prefill of a wide model
        {"name": "norm 16384 tokens", "op": "norm", "M": 16384, "K": 4096, "x": "bf16", "fmt": "mxfp8"},
        # one decoded token through one projection
        {"name": "product 1 token", "op": "product", "M": 1, "N": 1408, "K": 2048, "x": "mxfp8", "y": "f16"},
        # a 16-token speculative-verify batch through a wide projection: the weights' bytes count
        {"name": "product 16 tokens", "op": "product", "M": 16, "N": 8192, "K": 8192, "x": "mxfp8", "y": "bf16"},
        # the prefill batch through one projection: too few tiles to fill the card
        {"name": "product 512 tokens", "op": "product", "M": 512, "N": 1408, "K": 2048, "x": "mxfp8", "y": "bf16"},
        # odd numbers of tokens and outputs, a ragged reduction, 32-bit result (logits)
        {"name": "product ragged", "op": "product", "M": 333, "N": 4099, "K": 1440, "x": "mxfp4", "y": "f32"},
        # a 2048-token stack layer through the shared expert's gate and up
        {"name": "product 2048 tokens", "op": "product", "M": 2048, "N": 11264, "K": 2048, "x": "mxfp8", "y": "bf16"},
        # a large square product, both sides in 4 bits: the tensor cores' rate counts
        {"name": "product 8192", "op": "product", "M": 8192, "N": 8192, "K": 8192, "x": "mxfp4", "y": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["quantize", "norm", "product", "product"])
    if op == "quantize":
        return {"op": op, "M": _log(rng, 1, 16384), "K": 32 * _log(rng, 1, 256), "x": rng.choice(["bf16", "f16", "f32"]),
                "fmt": rng.choice(["mxfp8", "mxfp4"])}
    if op == "norm":
        return {"op": op, "M": _log(rng, 1, 8192), "K": 32 * _log(rng, 8, 256), "x": rng.choice(["bf16", "f16"]),
                "fmt": rng.choice(["mxfp8", "mxfp8", "mxfp4"])}
    return {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 8, 8192), "K": 32 * _log(rng, 8, 256),
            "x": rng.choice(["mxfp8", "mxfp4"]), "y": rng.choice(["bf16", "f16", "f32"])}


# ---- making inputs: seeded values, and codes and scales put together apart from what is measured

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _hidden(g, rows, cols):
    """Hidden states: unit normal, rows of differing size, some channels that stand out."""
    v = torch.randn((rows, cols), generator=g, device=DEV)
    v *= torch.exp(0.5 * torch.randn((rows, 1), generator=g, device=DEV))
    v *= torch.where(torch.rand((1, cols), generator=g, device=DEV) < 0.01, 8.0, 1.0)
    return v


def _random_mx(g, rows, K, fmt, spread):
    """Codes and tiled scales as a quantiser leaves them: uniform mantissas, the scales within `spread` binades."""
    nb = K // 32
    n = rows * K if fmt == "mxfp8" else rows * K // 2
    codes = torch.randint(0, 256, (n,), generator=g, device=DEV, dtype=torch.uint8)
    if fmt == "mxfp8":
        # magnitudes up to 448, most of them within six binades of it, and no NaN code
        mag = 126 - (torch.randn(n, generator=g, device=DEV).abs() * 20).to(torch.uint8).clamp_(max=126)
        codes = (codes & 128) | mag
    codes = codes.view(rows, -1)
    scales = torch.zeros((-(-rows // 128) * 128, -(-nb // 4) * 4), device=DEV, dtype=torch.uint8)
    scales[:rows, :nb] = torch.randint(119 - spread, 119, (rows, nb), generator=g, device=DEV, dtype=torch.uint8)
    tiles = scales.view(scales.shape[0] // 128, 4, 32, scales.shape[1] // 4, 4).permute(0, 3, 2, 1, 4)
    return codes, tiles.reshape(-1).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": dict(case)}
    M, K = case["M"], case["K"]
    if case["op"] == "product":
        st["x_codes"], st["x_scales"] = _random_mx(g, M, K, case["x"], 6)
        st["w_codes"], st["w_scales"] = _random_mx(g, case["N"], K, "mxfp4", 3)
    else:
        st["x"] = _hidden(g, M, K).to(DT[case["x"]])
        if case["op"] == "norm":
            st["residual"] = (3 * _hidden(g, M, K)).to(DT[case["x"]])
            st["weight"] = (1 + 0.2 * torch.randn(K, generator=g, device=DEV)).to(DT[case["x"]])
    return st


# ---- the plain forms

def _power(s):
    """2^(s - 127) of scale bytes s, in 32 bits; 255 is NaN."""
    s = s.to(torch.int32)
    p = torch.where(s == 0, torch.full_like(s, 0x00400000), s << 23).view(torch.float32)
    return torch.where(s == 255, torch.full_like(p, float("nan")), p)


def _plain_quantize(v, fmt):
    """[R, K] in 32 bits -> the values that codes and scales stand for [R, K], scale bytes [R, K / 32]."""
    R, K = v.shape
    v = v.view(R, K // 32, 32)
    big = v.abs().amax(-1)
    e = torch.frexp(big)[1] - 1 - EMAX[fmt]
    s = torch.where(big > 0, (e + 127).clamp(0, 254), torch.zeros_like(e))
    scale = _power(s)[..., None]
    a = (v / scale).abs()
    if fmt == "mxfp8":
        a = a.clamp(max=448.0)
        step = _power((torch.frexp(a)[1] - 1).clamp(min=-6) - 3 + 127)
    else:
        a = a.clamp(max=6.0)
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.copysign(torch.round(a / step) * step, v)
    return (q * scale).view(R, K), s.to(torch.uint8)


def _plain_values(codes, scales, fmt, K):
    """The values of an MX tensor in 32 bits."""
    R = codes.shape[0]
    if fmt == "mxfp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
        v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).view(R, K)
    t = scales.view(-(-R // 128), -(-K // 128), 32, 4, 4).permute(0, 3, 2, 1, 4)
    s = t.reshape(t.shape[0] * 128, -1)[:R, : K // 32]
    return (v.view(R, K // 32, 32) * _power(s)[..., None]).view(R, K)


def run(state):
    c = state["case"]
    if own:
        from int4_block_quantized_gb300 import binding as B
        fmt = {"mxfp8": B.MXFP8, "mxfp4": B.MXFP4}
        if c["op"] == "quantize":
            codes, scales = B.qmoe_mx_quantize(state["x"], fmt[c["fmt"]])
            return {"values": B.qmoe_mx_dequant(codes, scales, fmt[c["fmt"]], state["x"].dtype)}
        if c["op"] == "norm":
            codes, scales, total = B.qmoe_rmsnorm_mx(state["x"], state["residual"], state["weight"], EPS, fmt[c["fmt"]])
            return {"residual": total, "values": B.qmoe_mx_dequant(codes, scales, fmt[c["fmt"]], torch.bfloat16)}
        return {"y": B.qmoe_mx_matmul(state["x_codes"], state["x_scales"], fmt[c["x"]], state["w_codes"],
                                      state["w_scales"], DT[c["y"]])}
    if c["op"] == "quantize":
        return {"values": _plain_quantize(state["x"].float(), c["fmt"])[0].to(state["x"].dtype)}
    if c["op"] == "norm":
        h = state["x"].float() + state["residual"].float()
        y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * state["weight"].float()
        return {"residual": h.to(state["x"].dtype), "values": _plain_quantize(y, c["fmt"])[0].to(torch.bfloat16)}
    x = _plain_values(state["x_codes"], state["x_scales"], c["x"], c["K"])
    w = _plain_values(state["w_codes"], state["w_scales"], "mxfp4", c["K"])
    return {"y": (x @ w.t()).to(DT[c["y"]])}


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "product":
        N = case["N"]
        b = M * K * (1 if case["x"] == "mxfp8" else 0.5) + N * K * 0.5 + (M + N) * K / 32 + M * N * SIZE[case["y"]]
        return {"bytes": b, "flops": 2 * M * N * K}
    mx = M * K * ((1 if case["fmt"] == "mxfp8" else 0.5) + 1 / 32)
    if case["op"] == "quantize":  # x in, codes and scales out and in again, values out
        return {"bytes": 2 * M * K * SIZE[case["x"]] + 2 * mx, "flops": 4 * M * K}
    return {"bytes": 3 * M * K * 2 + K * 2 + 2 * mx + M * K * 2, "flops": 8 * M * K}


# ---- the definitions in 64 bits, from the list of values that a format has

def _grid(fmt):
    if fmt == "mxfp4":
        return [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    return [m / 512 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]


def _double_power(e):
    """2^e from the bits (a logarithm or a power function may miss a power of two by its last bit)."""
    return ((e + 1023) << 52).view(torch.float64)


def _exact_quantize(v, fmt):
    """Nearest value of the format, an exact middle to the one with the even code; in pieces of rows."""
    grid = torch.tensor(_grid(fmt), dtype=torch.float64, device=v.device)
    middle = (grid[1:] + grid[:-1]) / 2
    out = torch.empty_like(v)
    step = max(1, (1 << 24) // v.shape[1])
    for r in range(0, v.shape[0], step):
        b = v[r:r + step].reshape(-1, 32)
        big = b.abs().max(1, keepdim=True).values
        X = _double_power((torch.frexp(big)[1].long() - 1 - EMAX[fmt]).clamp(min=-127))
        a = b.abs() / X
        below = torch.bucketize(a, middle)               # middles strictly below a
        above = torch.bucketize(a, middle, right=True)   # middles at or below a
        code = torch.where((below != above) & (below % 2 == 1), above, below)
        out[r:r + step] = (grid[code] * torch.sign(b) * X).reshape(-1, v.shape[1])
    return out


def _exact_values(codes, scales, fmt, K):
    R, grid = codes.shape[0], torch.tensor(_grid(fmt), dtype=torch.float64, device=codes.device)
    if fmt == "mxfp8":
        mag, neg = codes.long() & 127, codes.long() >> 7
    else:
        both = torch.empty((R, K), dtype=torch.long, device=codes.device)
        both[:, 0::2], both[:, 1::2] = codes.long() % 16, codes.long() // 16
        mag, neg = both % 8, both // 8
    r = torch.arange(R, device=codes.device)[:, None]
    b = torch.arange(K // 32, device=codes.device)[None, :]
    at = (r // 128 * (-(-K // 128)) + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4
    X = _double_power(scales[at].long() - 127)
    return grid[mag] * (1 - 2 * neg) * X.repeat_interleave(32, 1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quantize":
        return {"values": _exact_quantize(st["x"].double(), case["fmt"])}
    if case["op"] == "norm":
        h = st["x"].double() + st["residual"].double()
        y = h / torch.sqrt(h.square().sum(1, keepdim=True) / case["K"] + EPS) * st["weight"].double()
        return {"residual": h, "values": _exact_quantize(y, case["fmt"])}
    x = _exact_values(st["x_codes"], st["x_scales"], case["x"], case["K"])
    w = _exact_values(st["w_codes"], st["w_scales"], "mxfp4", case["K"])
    return {"y": torch.einsum("mk,nk->mn", x, w)}
