"""The package offers the FP8 experts' calls as it does the others (no GPU)."""
import pytest

import int4_block_quantized_gb300 as package
from int4_block_quantized_gb300 import binding


@pytest.mark.parametrize("name", ["qmoe_fp8_quantize", "qmoe_fp8_quantize_swiglu", "qmoe_fp8_quantize_weights", "qmoe_fp8_dequant",
                                  "qmoe_fp8_matmul", "qmoe_fp8_status", "qmoe_sort_experts", "qmoe_dispatch", "qmoe_dispatch_backward",
                                  "qmoe_combine", "qmoe_combine_backward"])
def test_the_package_has(name):
    assert getattr(package, name) is getattr(binding, name)
