"""GPTQ per-layer quantization on MI355X (gfx950): HIP kernels behind the C ABI of libgptq_mi355x.so.

The Python layer only marshals arguments; see include/gptq_mi355x.h for the ABI,
include/gptq_mi355x_mx.h for the MX (microscaled) operators, and
include/gptq_mi355x_int8.h for those on 8-bit integers and the norm.
"""
from ._lib import (  # noqa: F401
    GPTQ_BF16, GPTQ_F32, GPTQ_FACTOR_INVERSE_RECHOL, GPTQ_FACTOR_R_FORM, GPTQ_FACTOR_REVERSED, GPTQ_GRID_ASYMMETRIC,
    GPTQ_GRID_SYMMETRIC, GPTQ_MX_E2M1, GPTQ_MX_E4M3, GPTQ_NORM_E4M3, GPTQ_NORM_INT8, GPTQError, LIB_PATH, load,
    status_string,
)
from .gptq import (  # noqa: F401
    HessianState, QuantizedLayer, QuantResult, apply_layerwise, dequant_matmul, factor_route, gptq_quantize,
    hessian_accumulate, pack_codes, prepare_chol, quantize_layer,
)
from .int8 import (  # noqa: F401
    Int8Tensor, int8_dequantize, int8_linear, int8_matmul, int8_quantize, int8_weight,
)
from .mx import (  # noqa: F401
    MXTensor, mx_dequantize, mx_grad_input, mx_grad_weight, mx_linear, mx_matmul, mx_quantize,
)
from .norm import NormResult, rms_norm, rms_norm_grad  # noqa: F401
