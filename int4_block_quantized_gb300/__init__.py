"""INT4 block-quantized mixture-of-experts FFN layer for NVIDIA GB300 (sm_103a).

The compute lives in a C-ABI CUDA library (csrc/, header include/qmoe.h);
`binding` is a thin ctypes layer over it with the same entry-point names.
Importing the package does not load the library; the binding does, and it
raises if the library is missing -- there is no CPU fallback.
"""

__all__ = ["binding", "synthetic"]


def __getattr__(name):
    if name in ("qmoe_route", "matmul_nbits", "qmoe_forward", "qmoe_dequant", "qmoe_rmsnorm",
                "qmoe_workspace_size", "qmoe_status_string", "QMoEError", "Workspace",
                "qmoe_mx_quantize", "qmoe_mx_dequant", "qmoe_rmsnorm_mx", "qmoe_mx_matmul",
                "qmoe_mx_tile_scales", "qmoe_mx_untile_scales", "qmoe_mx_scale_bytes", "qmoe_mx_status", "MXFP8", "MXFP4",
                "qmoe_fp8_quantize", "qmoe_fp8_quantize_swiglu", "qmoe_fp8_quantize_weights", "qmoe_fp8_dequant",
                "qmoe_fp8_matmul", "qmoe_fp8_status", "qmoe_sort_experts", "qmoe_dispatch", "qmoe_dispatch_backward",
                "qmoe_combine", "qmoe_combine_backward"):
        from . import binding
        return getattr(binding, name)
    raise AttributeError(name)
