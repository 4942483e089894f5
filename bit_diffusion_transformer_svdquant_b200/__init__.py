"""B200 (sm_100a) SVDQuant-style W4A4 + low-rank linear layer.

The layer ("Bringing Nunchaku 4-bit diffusion inference to Diffusers", "SVDQuant deep dive"):
4-bit NVFP4 weights and activations, outliers absorbed by a 16-bit low-rank branch W = L1 L2 + R,
the branch's down-projection fused with activation quantization and its up-projection fused with
the 4-bit GEMM. The compute lives in libsvdq.so (C ABI in include/svdq.h); this package is its thin
Python binding plus the seeded synthetic workloads and an offline weight-preparation helper.
"""
from ._lib import (EPI_BIAS, EPI_BIAS_SWIGLU, EPI_NONE, EPI_SWIGLU, Fp8rAct, Fp8rWeight, MxAct, MxWeight, Norm,
                   PackedWeight, QuantizedAct, SvdqError, block_norm, calibrate_act, dequantize_act_mx, device_status,
                   export_act, export_act_fp8r, export_act_mx, export_weight, export_weight_fp8r, export_weight_mx,
                   gated_residual, gated_residual_quantize_mx, gemm, gemm_fp8r, gemm_mx, gemm_swiglu_quant, linear,
                   linear_fp8r, linear_mx, mlp, mlp_mx, norm_quantize_act_mx, quantize_act, quantize_act_fp8r,
                   quantize_act_mx, set_wait_limit_ns, watchdog_selftest)

__all__ = ["EPI_BIAS", "EPI_BIAS_SWIGLU", "EPI_NONE", "EPI_SWIGLU", "Fp8rAct", "Fp8rWeight", "MxAct", "MxWeight",
           "Norm", "PackedWeight", "QuantizedAct", "SvdqError", "block_norm", "calibrate_act", "dequantize_act_mx",
           "device_status", "export_act", "export_act_fp8r", "export_act_mx", "export_weight", "export_weight_fp8r",
           "export_weight_mx", "gated_residual", "gated_residual_quantize_mx", "gemm", "gemm_fp8r", "gemm_mx",
           "gemm_swiglu_quant", "linear", "linear_fp8r", "linear_mx", "mlp", "mlp_mx", "norm_quantize_act_mx",
           "quantize_act", "quantize_act_fp8r", "quantize_act_mx", "set_wait_limit_ns", "watchdog_selftest"]
