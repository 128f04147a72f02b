"""Thin Python binding of the C ABI (include/qmoe.h) over ctypes.

Argument marshalling only: every step of the layer runs in the CUDA library
libqmoe.so.  Tensors are torch CUDA tensors (device memory and streams come
from PyTorch); calls are enqueued on torch's current stream.  There is no
fallback: if the library is missing this module raises on import use.
"""
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqmoe.so")

F16, BF16 = 0, 1
PATH_AUTO, PATH_DECODE, PATH_PREFILL, PATH_DECODE_SPLIT, PATH_DECODE_FUSED = 0, 1, 2, 4, 5
DECODE_MAX_TOKENS = 16
AUTO_DECODE_MAX_TOKENS = 5
DIAG_STALL_GEMM = 1
F32 = 2                      # the microscaled entry points that say so
MXFP8, MXFP4 = 0, 1
DIAG_STALL_FP8_CODES, DIAG_STALL_FP8_SCALES, DIAG_STALL_FP8_MMA, DIAG_STALL_FP8_OUTPUT = 1, 2, 4, 8
DIAG_STALL_MX_CODES, DIAG_STALL_MX_SCALES, DIAG_STALL_MX_MMA, DIAG_STALL_MX_OUTPUT, DIAG_STALL_MX_SPREAD = 1, 2, 4, 8, 16
_STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported device or shape",
           3: "workspace missing or too small", 4: "CUDA runtime error",
           5: "device wait timed out", 6: "device index check failed"}


class QMoEError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__("%s: %s (status %d)" % (where, _STATUS.get(code, "unknown"), code))


class QWeight(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("zp", ctypes.c_void_p)]


_lib = None


def lib():
    """The loaded libqmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libqmoe.so not built (run int4_block_quantized_gb300/build.py); "
                               "there is no CPU fallback")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.qmoe_status_string.restype = ctypes.c_char_p
        L.qmoe_status_string.argtypes = [i32]
        L.qmoe_last_cuda_error.restype = ctypes.c_char_p
        L.qmoe_last_cuda_error.argtypes = []
        L.qmoe_workspace_size.restype = sz
        L.qmoe_workspace_size.argtypes = [i32] * 5
        L.qmoe_workspace_init.restype = i32
        L.qmoe_workspace_init.argtypes = [vp, sz, vp]
        L.qmoe_workspace_set_diagnostics.restype = i32
        L.qmoe_workspace_set_diagnostics.argtypes = [vp, sz, ctypes.c_uint32, ctypes.c_uint32, vp]
        L.qmoe_route.restype = i32
        L.qmoe_route.argtypes = [vp, vp, i32, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
        L.matmul_nbits.restype = i32
        L.matmul_nbits.argtypes = [vp, i32, vp, vp, i32, vp, i32, i32, i32, i32, vp, vp]
        L.matmul_nbits_ex.restype = i32
        L.matmul_nbits_ex.argtypes = [vp, i32, vp, vp, i32, vp, i32, i32, i32, i32, vp, i32, vp, sz, vp]
        L.qmoe_forward.restype = i32
        L.qmoe_forward.argtypes = [vp, i32, vp, vp, QWeight, QWeight, QWeight] + [i32] * 7 + \
            [vp, vp, vp, i32, vp, sz, vp]
        L.qmoe_forward_ex.restype = i32
        L.qmoe_forward_ex.argtypes = [vp, i32, vp, vp, QWeight, QWeight, QWeight] + [i32] * 7 + \
            [vp, vp, vp, i32, i32, vp, sz, vp]
        L.qmoe_forward_kernels.restype = i32
        L.qmoe_forward_kernels.argtypes = [i32] * 11
        L.qmoe_forward_profiled.restype = i32
        L.qmoe_forward_profiled.argtypes = [vp, i32, vp, vp, QWeight, QWeight, QWeight] + [i32] * 7 + \
            [vp, i32, vp, sz, vp, ctypes.POINTER(ctypes.c_void_p), i32]
        L.qmoe_forward_noalloc.restype = i32
        L.qmoe_forward_noalloc.argtypes = [vp, i32, vp, vp, QWeight, QWeight, QWeight] + [i32] * 7 + \
            [vp, vp, vp, i32, vp]
        L.qmoe_noalloc_status.restype = i32
        L.qmoe_noalloc_status.argtypes = [ctypes.POINTER(ctypes.c_uint32), vp]
        L.qmoe_shared_expert.restype = i32
        L.qmoe_shared_expert.argtypes = [vp, i32, vp, QWeight, QWeight, QWeight] + [i32] * 5 + \
            [vp, i32, vp, sz, vp]
        L.qmoe_dequant.restype = i32
        L.qmoe_dequant.argtypes = [vp, vp, i32, vp, i32, i32, i32, vp, vp]
        L.qmoe_rmsnorm.restype = i32
        L.qmoe_rmsnorm.argtypes = [vp, vp, i32, i32, i32, ctypes.c_float, vp]
        L.qmoe_repack_gptq.restype = i32
        L.qmoe_repack_gptq.argtypes = [vp, vp, vp] + [i32] * 5 + [vp, vp, vp, vp, vp, vp]
        L.qmoe_gptq_zero_offset.restype = i32
        L.qmoe_gptq_zero_offset.argtypes = [vp, sz, vp, vp]
        L.qmoe_unpack_zero_points.restype = i32
        L.qmoe_unpack_zero_points.argtypes = [vp, i32, i32, vp, vp]
        L.qmoe_mx_scale_bytes.restype = sz
        L.qmoe_mx_scale_bytes.argtypes = [i32, i32]
        L.qmoe_mx_quantize.restype = i32
        L.qmoe_mx_quantize.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp]
        L.qmoe_mx_dequant.restype = i32
        L.qmoe_mx_dequant.argtypes = [vp, vp, i32, i32, i32, vp, i32, vp]
        L.qmoe_rmsnorm_mx.restype = i32
        L.qmoe_rmsnorm_mx.argtypes = [vp, vp, vp, i32, i32, i32, ctypes.c_float, i32, vp, vp, vp, vp]
        L.qmoe_mx_matmul.restype = i32
        L.qmoe_mx_matmul.argtypes = [vp, vp, i32, vp, vp, i32, i32, i32, vp, i32, vp, vp]
        L.qmoe_mx_matmul_diagnosed.restype = i32
        L.qmoe_mx_matmul_diagnosed.argtypes = [vp, vp, i32, vp, vp, i32, i32, i32, vp, i32, vp, ctypes.c_uint32,
                                               ctypes.c_uint32, vp]
        L.qmoe_mx_matmul_variant.restype = i32
        L.qmoe_mx_matmul_variant.argtypes = [i32, vp, i32, i32, i32, ctypes.POINTER(ctypes.c_int)]
        L.qmoe_mx_status.restype = i32
        L.qmoe_mx_status.argtypes = [ctypes.POINTER(ctypes.c_uint32), vp]
        for f in (L.qmoe_mx_tile_scales, L.qmoe_mx_untile_scales):
            f.restype = i32
            f.argtypes = [vp, i32, i32, vp, vp]
        L.qmoe_fp8_quantize.restype = i32
        L.qmoe_fp8_quantize.argtypes = [vp, i32, i32, i32, vp, i32, vp, vp, vp]
        L.qmoe_fp8_quantize_swiglu.restype = i32
        L.qmoe_fp8_quantize_swiglu.argtypes = [vp, i32, i32, i32, vp, vp, vp]
        L.qmoe_fp8_quantize_weights.restype = i32
        L.qmoe_fp8_quantize_weights.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp]
        L.qmoe_fp8_dequant.restype = i32
        L.qmoe_fp8_dequant.argtypes = [vp, vp, i32, i32, i32, i32, vp, i32, vp]
        L.qmoe_fp8_matmul.restype = i32
        L.qmoe_fp8_matmul.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, i32, vp, vp]
        L.qmoe_fp8_matmul_diagnosed.restype = i32
        L.qmoe_fp8_matmul_diagnosed.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, i32, vp, ctypes.c_uint32,
                                                ctypes.c_uint32, vp]
        L.qmoe_fp8_matmul_variant.restype = i32
        L.qmoe_fp8_matmul_variant.argtypes = [i32, i32, i32, i32, i32, ctypes.POINTER(ctypes.c_int)]
        L.qmoe_fp8_status.restype = i32
        L.qmoe_fp8_status.argtypes = [ctypes.POINTER(ctypes.c_uint32), vp]
        L.qmoe_sort_experts.restype = i32
        L.qmoe_sort_experts.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp]
        L.qmoe_dispatch.restype = i32
        L.qmoe_dispatch.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp]
        L.qmoe_dispatch_backward.restype = i32
        L.qmoe_dispatch_backward.argtypes = [vp, i32, vp, i32, i32, i32, vp, vp]
        L.qmoe_combine.restype = i32
        L.qmoe_combine.argtypes = [vp, i32, vp, vp, vp, i32, i32, i32, vp, i32, vp]
        L.qmoe_combine_backward.restype = i32
        L.qmoe_combine_backward.argtypes = [vp, i32, vp, i32, vp, vp, i32, i32, i32, vp, vp, vp]
        L.qmoe_get_device_status.restype = i32
        L.qmoe_get_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32), vp]
        _lib = L
    return _lib


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dt(t):
    return BF16 if t.dtype == torch.bfloat16 else F16


def _check(rc, where):
    if rc != 0:
        if rc == 4:
            where = "%s [%s]" % (where, lib().qmoe_last_cuda_error().decode())
        raise QMoEError(rc, where)


def qmoe_status_string(code):
    return lib().qmoe_status_string(code).decode()


def qmoe_workspace_size(T, H, I, E, k):
    return int(lib().qmoe_workspace_size(T, H, I, E, k))


class Workspace:
    """Caller-owned device workspace sized for (T, H, I, E, k), initialised once."""

    def __init__(self, T, H, I, E, k, device=None):
        self.nbytes = qmoe_workspace_size(T, H, I, E, k)
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device or "cuda")
        _check(lib().qmoe_workspace_init(_p(self.buf), self.nbytes, _stream()), "qmoe_workspace_init")

    @property
    def ptr(self):
        return ctypes.c_void_p(self.buf.data_ptr())

    def set_diagnostics(self, wait_limit_kilocycles=0, flags=0):
        """Diagnostics of the failure path: the grouped GEMM's waits give up
        after wait_limit_kilocycles x 1024 SM cycles (0: about 2 s); flags
        DIAG_STALL_GEMM makes its dequantisers wait for a copy that cannot
        arrive.  (0, 0) restores normal operation."""
        _check(lib().qmoe_workspace_set_diagnostics(self.ptr, self.nbytes, int(wait_limit_kilocycles), int(flags),
                                                    _stream()), "qmoe_workspace_set_diagnostics")

    def status(self):
        bits = ctypes.c_uint32(0)
        rc = lib().qmoe_get_device_status(self.ptr, ctypes.byref(bits), _stream())
        return rc, bits.value


def qmoe_route(x, router_w, k, router_bias=None, ws=None, grouping=True):
    """(topk_w [T,k] fp32, topk_ids [T,k] int32, offsets [E+1], perm [T*k])."""
    T, H = x.shape
    E = router_w.shape[1]
    ws = ws or Workspace(T, H, 32, E, k, device=x.device)
    tw = torch.empty((T, k), dtype=torch.float32, device=x.device)
    ti = torch.empty((T, k), dtype=torch.int32, device=x.device)
    off = torch.empty(E + 1, dtype=torch.int32, device=x.device) if grouping else None
    perm = torch.empty(T * k, dtype=torch.int32, device=x.device) if grouping else None
    _check(lib().qmoe_route(_p(x), _p(router_w), _dt(x), _p(router_bias), T, H, E, k, _p(tw), _p(ti),
                            _p(off), _p(perm), ws.ptr, ws.nbytes, _stream()), "qmoe_route")
    return tw, ti, off, perm


def matmul_nbits(x, w, scales, zp, block_size, out=None):
    """y[M,N] = x[M,K] . dequant(W)[N,K]^T for one packed [N, K/2] matrix."""
    M, K = x.shape
    N = w.shape[-2]
    y = out if out is not None else torch.empty((M, N), dtype=x.dtype, device=x.device)
    _check(lib().matmul_nbits(_p(x), _dt(x), _p(w), _p(scales), _dt(scales), _p(zp), M, N, K,
                              block_size, _p(y), _stream()), "matmul_nbits")
    return y


def matmul_nbits_ex(x, w, scales, zp, block_size, out=None, path=PATH_AUTO, ws=None):
    """matmul_nbits for any M: tensor cores above the decode token limit."""
    M, K = x.shape
    N = w.shape[-2]
    y = out if out is not None else torch.empty((M, N), dtype=x.dtype, device=x.device)
    ws = ws or Workspace(M, N, K, 1, 1, device=x.device)
    _check(lib().matmul_nbits_ex(_p(x), _dt(x), _p(w), _p(scales), _dt(scales), _p(zp), M, N, K,
                                 block_size, _p(y), path, ws.ptr, ws.nbytes, _stream()),
           "matmul_nbits_ex")
    return y


def _qw(L, p):
    return QWeight(L[p + "_w"].data_ptr(), L[p + "_s"].data_ptr(),
                   None if L.get(p + "_zp") is None else L[p + "_zp"].data_ptr())


def qmoe_forward(layer, x=None, out=None, ws=None, accumulate=False, path=PATH_AUTO,
                 return_routing=False):
    """The whole layer.  `layer` holds router_w, router_bias, gate_/up_/down_ w, s,
    zp (device tensors) and ints H, I, E, k, block_size; x [T, H] defaults to
    layer['x'].  Returns out [T, H] (and (topk_w, topk_ids) if asked)."""
    L = layer
    x = L["x"] if x is None else x
    T = x.shape[0]
    H, I, E, k, bs = (int(L[n]) for n in ("H", "I", "E", "k", "block_size"))
    ws = ws or Workspace(T, H, I, E, k, device=x.device)
    o = out if out is not None else torch.empty((T, H), dtype=x.dtype, device=x.device)
    tw = ti = None
    if return_routing:
        tw = torch.empty((T, k), dtype=torch.float32, device=x.device)
        ti = torch.empty((T, k), dtype=torch.int32, device=x.device)
    rc = lib().qmoe_forward_ex(_p(x), _dt(x), _p(L["router_w"]), _p(L.get("router_bias")),
                               _qw(L, "gate"), _qw(L, "up"), _qw(L, "down"), _dt(L["gate_s"]),
                               T, H, I, E, k, bs, _p(o), _p(tw), _p(ti), int(bool(accumulate)),
                               int(path), ws.ptr, ws.nbytes, _stream())
    _check(rc, "qmoe_forward")
    return (o, tw, ti) if return_routing else o


def qmoe_shared_expert(layer, x=None, out=None, ws=None, accumulate=False):
    """out (+)= sigmoid(x . shared_gate_w) * FFN(x) for a shared expert dict
    (make_shared_expert layout: E = 1 weights plus shared_gate_w [H])."""
    L = layer
    x = L["x"] if x is None else x
    T = x.shape[0]
    H, I, bs = (int(L[n]) for n in ("H", "I", "block_size"))
    ws = ws or Workspace(T, H, I, 1, 1, device=x.device)
    o = out if out is not None else torch.empty((T, H), dtype=x.dtype, device=x.device)
    rc = lib().qmoe_shared_expert(_p(x), _dt(x), _p(L["shared_gate_w"]), _qw(L, "gate"), _qw(L, "up"),
                                  _qw(L, "down"), _dt(L["gate_s"]), T, H, I, bs, _p(o),
                                  int(bool(accumulate)), ws.ptr, ws.nbytes, _stream())
    _check(rc, "qmoe_shared_expert")
    return o


def qmoe_forward_noalloc(layer, x=None, out=None, accumulate=False, return_routing=False):
    """qmoe_forward with the library's static device workspace (no caller
    workspace; calls on one device must not overlap)."""
    L = layer
    x = L["x"] if x is None else x
    T = x.shape[0]
    H, I, E, k, bs = (int(L[n]) for n in ("H", "I", "E", "k", "block_size"))
    o = out if out is not None else torch.empty((T, H), dtype=x.dtype, device=x.device)
    tw = ti = None
    if return_routing:
        tw = torch.empty((T, k), dtype=torch.float32, device=x.device)
        ti = torch.empty((T, k), dtype=torch.int32, device=x.device)
    rc = lib().qmoe_forward_noalloc(_p(x), _dt(x), _p(L["router_w"]), _p(L.get("router_bias")),
                                    _qw(L, "gate"), _qw(L, "up"), _qw(L, "down"), _dt(L["gate_s"]),
                                    T, H, I, E, k, bs, _p(o), _p(tw), _p(ti), int(bool(accumulate)),
                                    _stream())
    _check(rc, "qmoe_forward_noalloc")
    return (o, tw, ti) if return_routing else o


def qmoe_noalloc_status():
    """(status code, raw bits) of the static scratch's device status word on
    the current device; reads and clears it (synchronises the stream)."""
    bits = ctypes.c_uint32(0)
    rc = lib().qmoe_noalloc_status(ctypes.byref(bits), _stream())
    return rc, bits.value


def qmoe_forward_kernels(layer, T, path=PATH_AUTO):
    """Kernels one qmoe_forward call on this layer with T tokens launches on
    the current device (1 fused decode, 3 decode, 5 prefill)."""
    L = layer
    H, I, E, k, bs = (int(L[n]) for n in ("H", "I", "E", "k", "block_size"))
    n = lib().qmoe_forward_kernels(T, H, I, E, k, bs, _dt(L["router_w"]), _dt(L["gate_s"]),
                                   int(L.get("gate_zp") is not None), int(L.get("down_zp") is not None),
                                   int(path))
    if n < 0:
        _check(-n, "qmoe_forward_kernels")
    return n


def qmoe_forward_profiled(layer, events, x=None, out=None, ws=None, path=PATH_AUTO):
    """qmoe_forward that records torch.cuda.Event objects `events` before the
    first kernel and after each kernel (kernels serialised)."""
    L = layer
    x = L["x"] if x is None else x
    T = x.shape[0]
    H, I, E, k, bs = (int(L[n]) for n in ("H", "I", "E", "k", "block_size"))
    ws = ws or Workspace(T, H, I, E, k, device=x.device)
    o = out if out is not None else torch.empty((T, H), dtype=x.dtype, device=x.device)
    arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    rc = lib().qmoe_forward_profiled(_p(x), _dt(x), _p(L["router_w"]), _p(L.get("router_bias")),
                                     _qw(L, "gate"), _qw(L, "up"), _qw(L, "down"), _dt(L["gate_s"]),
                                     T, H, I, E, k, bs, _p(o), int(path), ws.ptr, ws.nbytes, _stream(),
                                     arr, len(events))
    _check(rc, "qmoe_forward_profiled")
    return o


def qmoe_dequant(w, scales, zp, block_size):
    """fp32 [N, K] = (q - zp) * scale of one packed [N, K/2] matrix."""
    N, K2 = w.shape[-2], w.shape[-1]
    out = torch.empty((N, 2 * K2), dtype=torch.float32, device=w.device)
    _check(lib().qmoe_dequant(_p(w), _p(scales), _dt(scales), _p(zp), N, 2 * K2, block_size, _p(out),
                              _stream()), "qmoe_dequant")
    return out


def qmoe_rmsnorm(x, eps=1e-6, out=None):
    T, H = x.shape
    o = out if out is not None else torch.empty_like(x)
    _check(lib().qmoe_rmsnorm(_p(x), _p(o), _dt(x), T, H, float(eps), _stream()), "qmoe_rmsnorm")
    return o


def qmoe_gptq_zero_offset(qzeros):
    """Device int32 [1]: 1 if the median stored GPTQ zero point is 7, else 0."""
    off = torch.empty(1, dtype=torch.int32, device=qzeros.device)
    _check(lib().qmoe_gptq_zero_offset(_p(qzeros), qzeros.numel(), _p(off), _stream()), "qmoe_gptq_zero_offset")
    return off


def qmoe_repack_gptq(qweight, qzeros, scales, block_size, zero_offset=0, zero_offset_dev=None, check=True,
                     status=None):
    """GPTQ (qweight [E, K/8, N] int32, qzeros [E, K/bs, N/8] int32 or None,
    scales [E, K/bs, N]) -> canonical (w [E, N, K/2] u8, scales [E, N, K/bs],
    zp [E, N, K/bs] u8 or None).  A zero point above 15 (stored 15 with
    offset 1) sets QMOE_ST_RANGE in the status word: with check=True (the
    default) this synchronises and raises QMoEError; with check=False the
    caller's own int32 device tensor `status` (if given) collects the bit."""
    E, K8, N = qweight.shape
    K = 8 * K8
    nb = K // block_size
    w = torch.empty((E, N, K // 2), dtype=torch.uint8, device=qweight.device)
    s = torch.empty((E, N, nb), dtype=scales.dtype, device=qweight.device)
    zp = torch.empty((E, N, nb), dtype=torch.uint8, device=qweight.device) if qzeros is not None else None
    st = status if status is not None else (torch.zeros(1, dtype=torch.int32, device=qweight.device) if check else None)
    _check(lib().qmoe_repack_gptq(_p(qweight), _p(qzeros), _p(scales), E, K, N, block_size, int(zero_offset),
                                  _p(zero_offset_dev), _p(w), _p(s), _p(zp), _p(st), _stream()), "qmoe_repack_gptq")
    if check and status is None:
        _check(lib().qmoe_get_device_status(_p(st), None, _stream()),
               "qmoe_repack_gptq (a GPTQ zero point above 15 does not fit the 4-bit format)")
    return w, s, zp


def qmoe_unpack_zero_points(zp_packed, nb):
    """[rows, ceil(nb/2)] packed zero points -> [rows, nb] uint8."""
    rows = zp_packed.shape[0]
    out = torch.empty((rows, nb), dtype=torch.uint8, device=zp_packed.device)
    _check(lib().qmoe_unpack_zero_points(_p(zp_packed), rows, nb, _p(out), _stream()), "qmoe_unpack_zero_points")
    return out


# ---- microscaled (MX) formats.  An MX tensor [R, K] is (codes, scales): codes
# uint8 [R, K] (MXFP8) or [R, K/2] (MXFP4), scales a flat uint8 tensor of
# qmoe_mx_scale_bytes(R, K) bytes in the tile order that qmoe.h defines.
# These calls check what they are given (CUDA, contiguous, one device, types
# and sizes) and run on the tensors' device, on torch's current stream there.
# A call's kernel takes a few microseconds at one token, so the host side is
# kept short: sizes worked out here, plain integers handed to ctypes, the
# stream's handle read without building a torch.cuda.Stream (2.9 us on the
# GB300's host cores), outputs from torch.empty (1.6 us; new_empty takes 3.4).

_U8 = torch.uint8
_MX_MAX = 1 << 30
_MX_DT = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}


def _bad(where, what):
    raise QMoEError(1, "%s: %s" % (where, what))


def _mx_size(t, where):
    """(rows, columns) of a 2-D tensor."""
    shape = t.shape
    if len(shape) != 2:
        _bad(where, "wants 2-D tensors, got %s" % (tuple(shape),))
    return shape


def _mx_check(t, dev, dtype, numel, where, name):
    """A contiguous tensor of a type and size on device dev, or an error."""
    if dev < 0 or t.get_device() != dev or t.dtype is not dtype or t.numel() != numel or not t.is_contiguous():
        _bad(where, "%s: wants %d contiguous %s on one CUDA device, got %s %s on %s%s" % (
            name, numel, dtype, tuple(t.shape), t.dtype, t.device, "" if t.is_contiguous() else ", not contiguous"))


def _mx_check2(t, dev, dtype, shape, where, name):
    """The same, for a tensor whose shape says which element is which."""
    if dev < 0 or t.get_device() != dev or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _bad(where, "%s: wants contiguous %s %s on one CUDA device, got %s %s on %s%s" % (
            name, tuple(shape), dtype, tuple(t.shape), t.dtype, t.device, "" if t.is_contiguous() else ", not contiguous"))


def _mx_bytes(R, K, where):
    """qmoe_mx_scale_bytes, with the library's limit on R and K: what is beyond
    32 bits would reach it as another size."""
    if R > _MX_MAX or K > _MX_MAX:
        raise QMoEError(2, "%s: [%d, %d], at most 2^30 rows and columns" % (where, R, K))
    return (R + 127) // 128 * ((K + 127) // 128) * 512 if R > 0 and K > 0 and K % 32 == 0 else 0


def _mx_out(R, K, fmt, x, dev, codes, scales, where):
    """(codes, scales) to write an MX tensor [R, K] to: the caller's, or new ones."""
    n = _mx_bytes(R, K, where)
    if n == 0 or (fmt != MXFP8 and fmt != MXFP4):
        _bad(where, "format %r, [%d, %d]: MXFP8 or MXFP4, rows and a multiple of 32 columns are wanted" % (fmt, R, K))
    cols = K >> fmt
    if codes is None:
        codes = torch.empty((R, cols), dtype=_U8, device=x.device)
    else:
        _mx_check2(codes, dev, _U8, (R, cols), where, "codes")
    if scales is None:
        scales = torch.empty(n, dtype=_U8, device=x.device)
    else:
        _mx_check(scales, dev, _U8, n, where, "scales")
    return codes, scales


def _mx_call(dev, fn, where, *args):
    """fn(*args, stream) on device dev and its current stream."""
    if dev == torch._C._cuda_getDevice():
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if rc:
        _check(rc, where)


def qmoe_mx_scale_bytes(R, K):
    """Bytes of the scale tiles of an MX tensor [R, K] (0 if it cannot be one)."""
    return (R + 127) // 128 * ((K + 127) // 128) * 512 if R > 0 and K > 0 and K % 32 == 0 else 0


def qmoe_mx_quantize(x, fmt=MXFP8, codes=None, scales=None):
    """(codes, scales) of x [M, K] (fp16, bf16 or fp32) in MXFP8 or MXFP4."""
    where = "qmoe_mx_quantize"
    M, K = _mx_size(x, where)
    dt, dev = _MX_DT.get(x.dtype), x.get_device()
    if dt is None or dev < 0 or not x.is_contiguous():
        _bad(where, "x: wants a contiguous CUDA tensor of fp16, bf16 or fp32, got %s on %s" % (x.dtype, x.device))
    codes, scales = _mx_out(M, K, fmt, x, dev, codes, scales, where)
    _mx_call(dev, lib().qmoe_mx_quantize, where, x.data_ptr(), dt, fmt, M, K, codes.data_ptr(), scales.data_ptr())
    return codes, scales


def qmoe_mx_dequant(codes, scales, fmt, dtype=torch.bfloat16, out=None):
    """[M, K] values (fp16, bf16 or fp32) of an MX tensor."""
    where = "qmoe_mx_dequant"
    M, K = _mx_size(codes, where)
    dt, dev = _MX_DT.get(dtype), codes.get_device()
    if dt is None or (fmt != MXFP8 and fmt != MXFP4):
        _bad(where, "unsupported output type %s or format %r" % (dtype, fmt))
    _mx_check(codes, dev, _U8, M * K, where, "codes")
    K <<= fmt
    _mx_check(scales, dev, _U8, _mx_bytes(M, K, where), where, "scales")
    if out is None:
        out = torch.empty((M, K), dtype=dtype, device=codes.device)
    else:
        _mx_check2(out, dev, dtype, (M, K), where, "out")
    _mx_call(dev, lib().qmoe_mx_dequant, where, codes.data_ptr(), scales.data_ptr(), fmt, M, K, out.data_ptr(), dt)
    return out


def qmoe_rmsnorm_mx(x, residual=None, weight=None, eps=1e-6, fmt=MXFP8, residual_out=None, codes=None, scales=None):
    """(codes, scales, residual_out) of RMSNorm(x + residual) * weight in MXFP8
    or MXFP4; residual_out = x + residual (a new tensor unless given; it may be
    x or residual itself).  Without a residual it is None unless given."""
    where = "qmoe_rmsnorm_mx"
    T, H = shape = _mx_size(x, where)
    dtype, dev = x.dtype, x.get_device()
    if dev < 0 or not x.is_contiguous() or (dtype is not torch.float16 and dtype is not torch.bfloat16):
        _bad(where, "x: wants a contiguous CUDA tensor of fp16 or bf16, got %s on %s" % (dtype, x.device))
    codes, scales = _mx_out(T, H, fmt, x, dev, codes, scales, where)
    rp = wp = op = None
    if residual is not None:
        _mx_check2(residual, dev, dtype, shape, where, "residual")
        rp = residual.data_ptr()
    if residual_out is not None:
        _mx_check2(residual_out, dev, dtype, shape, where, "residual_out")
        op = residual_out.data_ptr()
    elif residual is not None:
        residual_out = torch.empty_like(x)
        op = residual_out.data_ptr()
    if weight is not None:
        _mx_check(weight, dev, dtype, H, where, "weight")
        if weight.shape[-1] != H:  # [H], or [1, H] as broadcasting has it
            _bad(where, "weight: wants [%d], got %s" % (H, tuple(weight.shape)))
        wp = weight.data_ptr()
    _mx_call(dev, lib().qmoe_rmsnorm_mx, where, x.data_ptr(), rp, wp, _MX_DT[dtype], T, H, float(eps), fmt, op,
             codes.data_ptr(), scales.data_ptr())
    return codes, scales, residual_out


def qmoe_mx_matmul(x_codes, x_scales, x_fmt, w_codes, w_scales, dtype=torch.bfloat16, out=None, status=None,
                   diagnostics=None):
    """y [M, N] (fp16, bf16 or fp32) = x . W^T for an MX tensor x [M, K] and MXFP4
    weights W [N, K].  status: an int32 [1] device tensor that collects
    QMOE_ST_TIMEOUT (zero it first); without one qmoe_mx_status() tells.  diagnostics: (wait_limit_kilocycles,
    DIAG_STALL_MX_* flags) of qmoe_mx_matmul_diagnosed."""
    where = "qmoe_mx_matmul"
    M, K = _mx_size(x_codes, where)
    N, half = _mx_size(w_codes, where)
    dt, dev = _MX_DT.get(dtype), x_codes.get_device()
    if dt is None or (x_fmt != MXFP8 and x_fmt != MXFP4) or K << x_fmt != 2 * half:
        _bad(where, "x [%d, %d] bytes in format %r, W [%d, %d] bytes, result in %s" % (M, K, x_fmt, N, half, dtype))
    _mx_check(x_codes, dev, _U8, M * K, where, "x_codes")
    K = 2 * half
    _mx_check(x_scales, dev, _U8, _mx_bytes(M, K, where), where, "x_scales")
    _mx_check(w_codes, dev, _U8, N * half, where, "w_codes")
    _mx_check(w_scales, dev, _U8, _mx_bytes(N, K, where), where, "w_scales")
    if out is None:
        out = torch.empty((M, N), dtype=dtype, device=x_codes.device)
    else:
        _mx_check2(out, dev, dtype, (M, N), where, "out")
    st = None
    if status is not None:
        _mx_check(status, dev, torch.int32, 1, where, "status")
        st = status.data_ptr()
    if diagnostics is None:
        _mx_call(dev, lib().qmoe_mx_matmul, where, x_codes.data_ptr(), x_scales.data_ptr(), x_fmt, w_codes.data_ptr(),
                 w_scales.data_ptr(), M, N, K, out.data_ptr(), dt, st)
    else:
        _mx_call(dev, lib().qmoe_mx_matmul_diagnosed, where, x_codes.data_ptr(), x_scales.data_ptr(), x_fmt,
                 w_codes.data_ptr(), w_scales.data_ptr(), M, N, K, out.data_ptr(), dt, st, *diagnostics)
    return out


def qmoe_mx_matmul_variant(x_fmt, w_codes, M):
    """(tokens per tile, pairs of CTAs, CTAs along K, codes spread by warps) of
    the kernel that a product of M tokens with w_codes [N, K/2] runs."""
    where = "qmoe_mx_matmul_variant"
    N, half = _mx_size(w_codes, where)
    _mx_bytes(N, 2 * half, where), _mx_bytes(M, 2 * half, where)
    dev = w_codes.get_device()
    _mx_check(w_codes, dev, _U8, N * half, where, "w_codes")
    v = (ctypes.c_int * 4)()
    with torch.cuda.device(dev):
        _check(lib().qmoe_mx_matmul_variant(x_fmt, w_codes.data_ptr(), M, N, 2 * half, v), where)
    return tuple(v)


def qmoe_mx_status():
    """(code, bits) of the products on the current device that were given no
    status tensor, and cleared: code 5 where one of them timed out.  Waits for
    the current stream."""
    bits = ctypes.c_uint32(0)
    rc = lib().qmoe_mx_status(ctypes.byref(bits), _stream())
    if rc not in (0, 5):
        _check(rc, "qmoe_mx_status")
    return rc, bits.value


def qmoe_mx_tile_scales(scales_rowmajor):
    """Row-major scale bytes [R, K/32] (as checkpoints store them) -> tiles."""
    where = "qmoe_mx_tile_scales"
    R, nb = _mx_size(scales_rowmajor, where)
    dev, n = scales_rowmajor.get_device(), _mx_bytes(R, 32 * nb, where)
    if n == 0:
        _bad(where, "wants scales [R, K/32]")
    _mx_check(scales_rowmajor, dev, _U8, R * nb, where, "scales")
    out = torch.empty(n, dtype=_U8, device=scales_rowmajor.device)
    _mx_call(dev, lib().qmoe_mx_tile_scales, where, scales_rowmajor.data_ptr(), R, 32 * nb, out.data_ptr())
    return out


def qmoe_mx_untile_scales(scales, R, K):
    """Scale tiles of an MX tensor [R, K] -> row-major bytes [R, K/32]."""
    where = "qmoe_mx_untile_scales"
    dev, n = scales.get_device(), _mx_bytes(R, K, where)
    if n == 0:
        _bad(where, "no MX tensor is [%d, %d]" % (R, K))
    _mx_check(scales, dev, _U8, n, where, "scales")
    out = torch.empty((R, K // 32), dtype=_U8, device=scales.device)
    _mx_call(dev, lib().qmoe_mx_untile_scales, where, scales.data_ptr(), R, K, out.data_ptr())
    return out


# ---- FP8 tensors with a scale for each block of 128, and experts in that format.
# An FP8 tensor is (codes, scales): codes uint8 [M, K] (or [E, N, K], weights),
# scales fp32 [M, ceil(K/128)] ([E, ceil(N/128), ceil(K/128)]); qmoe.h has the
# formulas.  pos int32 [T, k] is each assignment's place in the experts' order
# (qmoe_sort_experts); rows that it does not name are left as they were, so a
# call that makes its own output leaves them undefined.  Checked and run like the
# microscaled calls above.

# Each tensor's check is written out where it passes and made again, by
# _mx_check2, where it does not, to say what is wrong (a call of _mx_check2 takes
# 0.3 us, and a product has six tensors).

_F32 = torch.float32
_I32 = torch.int32
_ROWS_MAX = 1 << 30


def _fp8_in(x, dev, where, name):
    """qmoe_dtype of a contiguous fp16, bf16 or fp32 tensor on device dev."""
    dt = _MX_DT.get(x.dtype)
    if dt is None or dev < 0 or x.get_device() != dev or not x.is_contiguous():
        _bad(where, "%s: wants a contiguous fp16, bf16 or fp32 tensor on one CUDA device, got %s on %s%s" % (
            name, x.dtype, x.device, "" if x.is_contiguous() else ", not contiguous"))
    return dt


def _fp8_size(rows, K, where):
    if rows > _ROWS_MAX or K > _ROWS_MAX:
        raise QMoEError(2, "%s: %d rows of %d, at most 2^30 of each" % (where, rows, K))
    if rows < 1 or K < 16 or K % 16:
        _bad(where, "%d rows of %d: rows and a multiple of 16 columns are wanted" % (rows, K))


def _fp8_out(codes, scales, shape, sshape, x, dev, where):
    """(codes, scales) to write to: the caller's, or new ones."""
    if codes is None:
        codes = torch.empty(shape, dtype=_U8, device=x.device)
    elif codes.get_device() != dev or codes.dtype is not _U8 or codes.shape != shape or not codes.is_contiguous():
        _mx_check2(codes, dev, _U8, shape, where, "codes")
    if scales is None:
        scales = torch.empty(sshape, dtype=_F32, device=x.device)
    elif scales.get_device() != dev or scales.dtype is not _F32 or scales.shape != sshape or not scales.is_contiguous():
        _mx_check2(scales, dev, _F32, sshape, where, "scales")
    return codes, scales


def _places(pos, T, dev, where):
    """k of pos [T, k], checked."""
    shape = pos.shape
    if len(shape) != 2 or shape[0] != T or shape[1] < 1:
        _bad(where, "pos: wants [%d, k], got %s" % (T, tuple(shape)))
    k = shape[1]
    if T * k > _ROWS_MAX:
        raise QMoEError(2, "%s: %d x %d assignments, at most 2^30" % (where, T, k))
    if pos.get_device() != dev or dev < 0 or pos.dtype is not _I32 or not pos.is_contiguous():
        _mx_check2(pos, dev, _I32, shape, where, "pos")
    return k


def qmoe_fp8_quantize(x, pos=None, codes=None, scales=None):
    """(codes, scales) of x [T, K] (fp16, bf16 or fp32).  With pos [T, k] they have
    T * k rows, and token t is written to each row pos[t, j]."""
    where = "qmoe_fp8_quantize"
    T, K = _mx_size(x, where)
    dev = x.get_device()
    dt = _MX_DT.get(x.dtype)
    if dt is None or dev < 0 or not x.is_contiguous():
        _fp8_in(x, dev, where, "x")
    rows, k, pp = T, 0, None
    if pos is not None:
        k = _places(pos, T, dev, where)
        rows, pp = T * k, pos.data_ptr()
    _fp8_size(rows, K, where)
    codes, scales = _fp8_out(codes, scales, (rows, K), (rows, (K + 127) // 128), x, dev, where)
    _mx_call(dev, lib().qmoe_fp8_quantize, where, x.data_ptr(), dt, T, K, pp, k, codes.data_ptr(), scales.data_ptr())
    return codes, scales


def qmoe_fp8_quantize_swiglu(h, codes=None, scales=None):
    """(codes, scales) of silu(gate) * up [M, I] for h = [gate | up] [M, 2 I]."""
    where = "qmoe_fp8_quantize_swiglu"
    M, I = _mx_size(h, where)
    dev = h.get_device()
    dt = _fp8_in(h, dev, where, "h")
    if I % 2:
        _bad(where, "h: wants gate and up side by side, got %d columns" % I)
    I //= 2
    _fp8_size(M, I, where)
    codes, scales = _fp8_out(codes, scales, (M, I), (M, (I + 127) // 128), h, dev, where)
    _mx_call(dev, lib().qmoe_fp8_quantize_swiglu, where, h.data_ptr(), dt, M, I, codes.data_ptr(), scales.data_ptr())
    return codes, scales


def qmoe_fp8_quantize_weights(w, codes=None, scales=None):
    """(codes, scales) of weights [E, N, K] or [N, K], a scale per 128 x 128."""
    where = "qmoe_fp8_quantize_weights"
    shape = tuple(w.shape)
    if len(shape) not in (2, 3):
        _bad(where, "w: wants [E, N, K] or [N, K], got %s" % (shape,))
    E, N, K = (1,) * (3 - len(shape)) + shape
    dev = w.get_device()
    dt = _fp8_in(w, dev, where, "w")
    _fp8_size(E * N, K, where)
    codes, scales = _fp8_out(codes, scales, shape, shape[:-2] + ((N + 127) // 128, (K + 127) // 128), w, dev, where)
    _mx_call(dev, lib().qmoe_fp8_quantize_weights, where, w.data_ptr(), dt, E, N, K, codes.data_ptr(), scales.data_ptr())
    return codes, scales


def qmoe_fp8_dequant(codes, scales, dtype=torch.bfloat16, out=None):
    """Values (fp16, bf16 or fp32) of an FP8 tensor; whether a scale covers one row
    or 128 is read from the scales' shape."""
    where = "qmoe_fp8_dequant"
    shape = codes.shape
    dims = len(shape)
    if dims not in (2, 3) or len(scales.shape) != dims:
        _bad(where, "codes %s with scales %s" % (tuple(shape), tuple(scales.shape)))
    N, K = shape[-2], shape[-1]
    E = shape[0] if dims == 3 else 1
    dev, dt = codes.get_device(), _MX_DT.get(dtype)
    if dt is None:
        _bad(where, "unsupported output type %s" % dtype)
    _fp8_size(E * N, K, where)
    if dev < 0 or codes.dtype is not _U8 or not codes.is_contiguous():
        _mx_check2(codes, dev, _U8, shape, where, "codes")
    rows = 1 if scales.shape[-2] == N else 128
    sshape = ((N + rows - 1) // rows, (K + 127) // 128) if dims == 2 else (E, (N + rows - 1) // rows, (K + 127) // 128)
    if scales.get_device() != dev or scales.dtype is not _F32 or scales.shape != sshape or not scales.is_contiguous():
        _mx_check2(scales, dev, _F32, sshape, where, "scales")
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=codes.device)
    else:
        _mx_check2(out, dev, dtype, shape, where, "out")
    _mx_call(dev, lib().qmoe_fp8_dequant, where, codes.data_ptr(), scales.data_ptr(), E, N, K, rows, out.data_ptr(), dt)
    return out


def qmoe_fp8_matmul(x_codes, x_scales, w_codes, w_scales, dtype=torch.bfloat16, offsets=None, out=None, status=None,
                    diagnostics=None):
    """y [M, N] (fp16, bf16 or fp32) = x . W^T for FP8 tensors x [M, K] and W [N, K];
    with offsets int32 [E + 1] and W [E, N, K], rows offsets[e] .. offsets[e + 1] - 1
    meet W[e], and the rows of y outside every expert's are left as they were.
    status: an int32 [1] device tensor that collects QMOE_ST_* bits (zero it
    first); without one qmoe_fp8_status() tells.  diagnostics: (wait_limit_kilocycles,
    DIAG_STALL_FP8_* flags) of qmoe_fp8_matmul_diagnosed."""
    where = "qmoe_fp8_matmul"
    M, K = _mx_size(x_codes, where)
    dev, dt = x_codes.get_device(), _MX_DT.get(dtype)
    shape = w_codes.shape
    op = st = None
    E = 1
    if offsets is not None:
        E = offsets.numel() - 1
        if offsets.get_device() != dev or offsets.dtype is not _I32 or len(offsets.shape) != 1 or not offsets.is_contiguous():
            _mx_check2(offsets, dev, _I32, (E + 1,), where, "offsets")
        op = offsets.data_ptr()
    dims = len(shape)
    N = shape[-2] if dims == 3 and shape[0] == E or dims == 2 and E == 1 else 0
    if dt is None or N < 1 or E < 1 or shape[-1] != K:
        _bad(where, "x %s, W %s, %s experts, result in %s" % (tuple(x_codes.shape), tuple(shape), E, dtype))
    if E > 256:
        raise QMoEError(2, "%s: %d experts, at most 256" % (where, E))
    _fp8_size(M, K, where)
    if E * N > _ROWS_MAX:
        _fp8_size(E * N, K, where)
    nb, rb = (K + 127) // 128, (N + 127) // 128
    sshape = (E, rb, nb) if dims == 3 else (rb, nb)
    if not (dev >= 0 and x_codes.dtype is _U8 and x_codes.is_contiguous() and
            x_scales.get_device() == dev and x_scales.dtype is _F32 and x_scales.shape == (M, nb) and x_scales.is_contiguous() and
            w_codes.get_device() == dev and w_codes.dtype is _U8 and w_codes.is_contiguous() and
            w_scales.get_device() == dev and w_scales.dtype is _F32 and w_scales.shape == sshape and w_scales.is_contiguous()):
        _mx_check2(x_codes, dev, _U8, (M, K), where, "x_codes")
        _mx_check2(x_scales, dev, _F32, (M, nb), where, "x_scales")
        _mx_check2(w_codes, dev, _U8, shape, where, "w_codes")
        _mx_check2(w_scales, dev, _F32, sshape, where, "w_scales")
    if out is None:
        out = torch.empty((M, N), dtype=dtype, device=x_codes.device)
    elif out.get_device() != dev or out.dtype is not dtype or out.shape != (M, N) or not out.is_contiguous():
        _mx_check2(out, dev, dtype, (M, N), where, "out")
    if status is not None:
        _mx_check(status, dev, _I32, 1, where, "status")
        st = status.data_ptr()
    if diagnostics is None:
        _mx_call(dev, lib().qmoe_fp8_matmul, where, x_codes.data_ptr(), x_scales.data_ptr(), w_codes.data_ptr(),
                 w_scales.data_ptr(), op, E, M, N, K, out.data_ptr(), dt, st)
    else:
        _mx_call(dev, lib().qmoe_fp8_matmul_diagnosed, where, x_codes.data_ptr(), x_scales.data_ptr(), w_codes.data_ptr(),
                 w_scales.data_ptr(), op, E, M, N, K, out.data_ptr(), dt, st, *diagnostics)
    return out


def qmoe_fp8_matmul_variant(M, N, K, E=None):
    """(tile, form, CTAs along K) of the kernel that a product of these sizes runs on
    the current device, as qmoe.h has them; E: grouped, over so many experts."""
    v = (ctypes.c_int * 3)()
    _fp8_size(M, K, "qmoe_fp8_matmul_variant"), _fp8_size(N * (E or 1), K, "qmoe_fp8_matmul_variant")
    _check(lib().qmoe_fp8_matmul_variant(E is not None, 1 if E is None else E, M, N, K, v), "qmoe_fp8_matmul_variant")
    return tuple(v)


def qmoe_fp8_status():
    """(code, bits) of the FP8 products on the current device that were given no
    status tensor, and cleared.  Waits for the current stream."""
    bits = ctypes.c_uint32(0)
    rc = lib().qmoe_fp8_status(ctypes.byref(bits), _stream())
    if rc not in (0, 5, 6):
        _check(rc, "qmoe_fp8_status")
    return rc, bits.value


def _fp8_wanted(t, shape, dtype, like, dev, where, name):
    """(output, its address): the caller's tensor, a new one for None, nothing for False."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=like.device)
    elif t is False:
        return None, None
    elif t.get_device() != dev or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _mx_check2(t, dev, dtype, shape, where, name)
    return t, t.data_ptr()


def qmoe_sort_experts(ids, E, offsets=None, perm=None, pos=None):
    """(offsets [E + 1], perm [T * k], pos [T, k]), int32, of ids int32 [T, k]: the
    assignments by expert, stably; an id outside 0 .. E - 1 goes nowhere (pos -1,
    and perm -1 behind the last).  An output that is given is written to; False: it
    is not wanted, and None stands in its place."""
    where = "qmoe_sort_experts"
    T, k = _mx_size(ids, where)
    dev = ids.get_device()
    if E > 256 or T * k > _ROWS_MAX:
        raise QMoEError(2, "%s: %d experts, %d assignments: at most 256 and 2^30" % (where, E, T * k))
    if E < 1 or T < 1 or k < 1:
        _bad(where, "ids %s, %d experts" % ((T, k), E))
    if dev < 0 or ids.dtype is not _I32 or not ids.is_contiguous():
        _mx_check2(ids, dev, _I32, (T, k), where, "ids")
    if offsets is perm is pos is None:  # (the usual call, without three calls of the helper)
        at = ids.device
        offsets = torch.empty((E + 1,), dtype=_I32, device=at)
        perm = torch.empty((T * k,), dtype=_I32, device=at)
        pos = torch.empty((T, k), dtype=_I32, device=at)
        po, pm, pp = offsets.data_ptr(), perm.data_ptr(), pos.data_ptr()
    else:
        offsets, po = _fp8_wanted(offsets, (E + 1,), _I32, ids, dev, where, "offsets")
        perm, pm = _fp8_wanted(perm, (T * k,), _I32, ids, dev, where, "perm")
        pos, pp = _fp8_wanted(pos, (T, k), _I32, ids, dev, where, "pos")
    _mx_call(dev, lib().qmoe_sort_experts, where, ids.data_ptr(), T, k, E, po, pm, pp)
    return offsets, perm, pos


def _fp8_rows(T, H, where):
    if T < 1 or H < 8 or H % 8:
        _bad(where, "[%d, %d]: rows and a multiple of 8 columns are wanted" % (T, H))
    if H > 1 << 28:
        raise QMoEError(2, "%s: %d columns, at most 2^28" % (where, H))


def qmoe_dispatch(x, pos, out=None):
    """xs [T * k, H] with xs[pos[t, j]] = x[t]."""
    where = "qmoe_dispatch"
    T, H = _mx_size(x, where)
    dev = x.get_device()
    dt = _fp8_in(x, dev, where, "x")
    _fp8_rows(T, H, where)
    k = _places(pos, T, dev, where)
    if out is None:
        out = torch.empty((T * k, H), dtype=x.dtype, device=x.device)
    elif out.get_device() != dev or out.dtype is not x.dtype or out.shape != (T * k, H) or not out.is_contiguous():
        _mx_check2(out, dev, x.dtype, (T * k, H), where, "out")
    _mx_call(dev, lib().qmoe_dispatch, where, x.data_ptr(), dt, T, H, k, pos.data_ptr(), out.data_ptr())
    return out


def _combine(where, ys, pos, w, residual, out):
    rows, H = _mx_size(ys, where)
    dev, yt = ys.get_device(), ys.dtype
    dt = _MX_DT.get(yt)
    if dt is None or dev < 0 or not ys.is_contiguous():
        _fp8_in(ys, dev, where, "ys")
    if len(pos.shape) != 2:
        _bad(where, "pos: wants [T, k], got %s" % (tuple(pos.shape),))
    T = pos.shape[0]
    _fp8_rows(T, H, where)
    k = _places(pos, T, dev, where)
    if rows != T * k:
        _bad(where, "ys: wants %d rows, got %d" % (T * k, rows))
    wp = rp = None
    if w is not None:
        if w.get_device() != dev or w.dtype is not _F32 or w.shape != (T, k) or not w.is_contiguous():
            _mx_check2(w, dev, _F32, (T, k), where, "w")
        wp = w.data_ptr()
    if residual is not None:
        yt = residual.dtype
        ot = _MX_DT.get(yt)
        if ot is None or residual.get_device() != dev or residual.shape != (T, H) or not residual.is_contiguous():
            _fp8_in(residual, dev, where, "residual")
            _mx_check2(residual, dev, yt, (T, H), where, "residual")
        rp = residual.data_ptr()
    elif out is not None:
        ot, yt = _fp8_in(out, dev, where, "out"), out.dtype
    else:
        ot = dt
    if out is None:
        out = torch.empty((T, H), dtype=yt, device=ys.device)
    elif out.get_device() != dev or out.dtype is not yt or out.shape != (T, H) or not out.is_contiguous():
        _mx_check2(out, dev, yt, (T, H), where, "out")
    _mx_call(dev, lib().qmoe_combine, where, ys.data_ptr(), dt, pos.data_ptr(), wp, rp, T, H, k, out.data_ptr(), ot)
    return out


def qmoe_combine(ys, pos, w=None, residual=None, out=None):
    """out [T, H] = residual + sum_j w[t, j] ys[pos[t, j]]: of the residual's type
    (without one, of out's or of ys').  w fp32 [T, k]; None: ones.  out may be
    residual."""
    return _combine("qmoe_combine", ys, pos, w, residual, out)


def qmoe_dispatch_backward(dxs, pos, out=None):
    """dx [T, H] = sum_j dxs[pos[t, j]], the gradient of qmoe_dispatch."""
    if out is not None and out.dtype is not dxs.dtype:
        _bad("qmoe_dispatch_backward", "out: wants %s, got %s" % (dxs.dtype, out.dtype))
    return _combine("qmoe_dispatch_backward", dxs, pos, None, None, out)


def qmoe_combine_backward(dout, ys, pos, w=None, dys=None, dw=None):
    """(dys [T * k, H], dw [T, k] fp32) of qmoe_combine for dout [T, H].  A gradient
    that is given is written to; False: it is not wanted, and None stands in its
    place.  ys may be None where dw is not wanted (dys is then of dout's type, or as
    given).  Rows of a new dys that no place names are not initialised."""
    where = "qmoe_combine_backward"
    T, H = _mx_size(dout, where)
    dev = dout.get_device()
    dt = _fp8_in(dout, dev, where, "dout")
    _fp8_rows(T, H, where)
    k = _places(pos, T, dev, where)
    if dw is False and dys is False:
        _bad(where, "neither gradient is wanted")
    if ys is not None:
        yt = _fp8_in(ys, dev, where, "ys")
        if ys.shape != (T * k, H):
            _mx_check2(ys, dev, ys.dtype, (T * k, H), where, "ys")
        dtype, yp = ys.dtype, ys.data_ptr()
    elif dw is not False:
        _bad(where, "ys: wanted for dw")
    else:
        dtype, yp = (dout if dys is None else dys).dtype, None
        yt = dt if dys is None else _fp8_in(dys, dev, where, "dys")
    wp = None
    if w is not None:
        if w.get_device() != dev or w.dtype is not _F32 or w.shape != (T, k) or not w.is_contiguous():
            _mx_check2(w, dev, _F32, (T, k), where, "w")
        wp = w.data_ptr()
    dys, dp = _fp8_wanted(dys, (T * k, H), dtype, dout, dev, where, "dys")
    dw, dwp = _fp8_wanted(dw, (T, k), _F32, dout, dev, where, "dw")
    _mx_call(dev, lib().qmoe_combine_backward, where, dout.data_ptr(), dt, yp, yt, pos.data_ptr(), wp, T, H, k, dp, dwp)
    return dys, dw
