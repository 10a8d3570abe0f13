"""gemmf32 for MI355X: FP32 C = A.B through LDS tiles with single- and double-buffered
K-loops, FP32 matrix-core micro-kernels and a measured per-shape dispatcher.

The compute path is the HIP library `libgemmf32.so` (C ABI in include/gemmf32.h); this
package only loads it and marshals arguments.  Next to the FP32 product it has 8-bit
block-scaled and expert-grouped products with their gradients (`lowp`, C ABI in
include/gemm_lp.h), and what a layer of experts needs around them: a router with its balance
loss, rows by expert, adapters of low rank, gated units and rows kept in 8 bits (`experts`, C ABI
in include/gemm_experts.h).  Build it with
`python -m tiled_double_buffered_amd.build`.
"""
from ._binding import (  # noqa: F401
    ERR_ALIAS, ERR_BAD_CONFIG, ERR_BAD_LD, ERR_BAD_TYPE, ERR_HIP, ERR_MISALIGNED, ERR_NEGATIVE_DIM,
    ERR_NULL_PTR, ERR_SCRATCH_LIMIT, ERR_TOO_LARGE, OK, SCRATCH_FLOATS, SIGNATURES,
    VARIANT_AUTO, VARIANT_DB, VARIANT_KS, VARIANT_MS, VARIANT_SB, VARIANT_SB3, GemmError,
    gemm_f32, gemm_f32_config_info, gemm_f32_config_ks, gemm_f32_config_ms,
    gemm_f32_config_variants, gemm_f32_db, gemm_f32_ex, gemm_f32_last_hip_error, gemm_f32_ms,
    gemm_f32_num_configs, gemm_f32_peak_probe, gemm_f32_sb, gemm_f32_select,
    gemm_f32_select_cfg, gemm_f32_splitk, gemm_f32_splitk_noalloc, gemm_f32_splitk_plan,
    gemm_f32_splitk_select, gemm_f32_splitk_workspace, gemm_f32_strerror, gemm_f32_version,
    load, matmul, matmul_splitk,
)

_LOWP = ("gemm_fp8", "gemm_fp8_exp", "gemm_fp8_quantize", "gemm_fp8_quantize_exp", "gemm_grouped", "gemm_grouped_wgrad", "linear_fp8",
         "linear_grouped", "matmul_fp8", "matmul_fp8_grouped", "matmul_grouped",
         "matmul_grouped_wgrad", "quantize_fp8", "quantize_fp8_pair")

_EXPERTS = ("add_adapters", "dequantize_fp8", "gated_silu", "gemm_adapters_down",
            "gemm_adapters_grad", "gemm_adapters_grad_workspace", "gemm_adapters_splits",
            "gemm_adapters_up", "gemm_fp8_dequantize", "gemm_gated", "gemm_gated_grad",
            "gemm_group_rows", "gemm_group_rows_workspace", "gemm_route", "gemm_route_grad",
            "gemm_route_workspace", "group_rows", "route_experts")


def __getattr__(name):
    # the low-precision and expert-grouped products and what is around them, loaded on first use:
    # they need torch, which the FP32 entry points import only when they are given tensors
    if name in _LOWP:
        from . import lowp
        globals()[name] = value = getattr(lowp, name)
        return value
    if name in _EXPERTS:
        from . import experts
        globals()[name] = value = getattr(experts, name)
        return value
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


def __dir__():
    return sorted({*globals(), *_LOWP, *_EXPERTS})


__version__ = "0.1.0"
