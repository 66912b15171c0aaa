"""B200 (sm_100a) QLoRA NF4 library: NF4 block-wise absmax quantization,
double quantization of the absmax constants, dequantization, the QLoRA linear
layer forward/backward, and microscaled (MX) 4-bit serving, behind the C ABI of
include/qlora.h.

The compute runs in ``libqlora_b200.so`` (hand-written CUDA); ``binding``
marshals torch tensors into it. Importing this package does not load the
library; the first call does, and fails loudly if it has not been built.
"""
from .binding import (MX_E2M1, MX_E4M3, MXTensor, NF4Weight, QloraError, load_library, qlora_dequantize_mx,
                      qlora_dequantize_nf4_dq, qlora_device_error, qlora_linear_bwd, qlora_linear_fwd,
                      qlora_mx_grouped_fwd, qlora_mx_linear_fwd, qlora_mx_storage_bytes, qlora_nf4_codebook,
                      qlora_nf4_storage_bytes, qlora_quantize_mx, qlora_quantize_nf4_dq, qlora_rmsnorm_mx,
                      qlora_status_string)

__all__ = ["MX_E2M1", "MX_E4M3", "MXTensor", "NF4Weight", "QloraError", "load_library", "qlora_dequantize_mx",
           "qlora_dequantize_nf4_dq", "qlora_device_error", "qlora_linear_bwd", "qlora_linear_fwd",
           "qlora_mx_grouped_fwd", "qlora_mx_linear_fwd", "qlora_mx_storage_bytes", "qlora_nf4_codebook",
           "qlora_nf4_storage_bytes", "qlora_quantize_mx", "qlora_quantize_nf4_dq", "qlora_rmsnorm_mx",
           "qlora_status_string"]
