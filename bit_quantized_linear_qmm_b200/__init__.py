"""Quantized linear layers on the NVIDIA B200 (sm_100a), computed straight from
packed low-bit weights.  The compute lives in libqlin.so (C ABI: include/qlin.h);
this package holds its sources (csrc/), its build script and a thin binding."""
from . import qlin  # noqa: F401
from .qlin import (  # noqa: F401
    AdapterPlan, QlinError, adapters_backward, adapters_forward, adapters_plan, adapters_workspace_size,
    bitlinear_matmul, dequantize, dequantize_int8_groups, device_status, int8_matmul_int32, matmul,
    pack_int4_cols, pergroup_linear, pergroup_wgrad, quantize, quantize_int8_groups, quantize_int8_rows,
    w4a8_linear, w8a8_linear, workspace_size,
)
