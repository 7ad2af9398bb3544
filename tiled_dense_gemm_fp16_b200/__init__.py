"""B200 (sm_100a) tiled fp16 GEMM with fused ReLU: C = ReLU(A . B).

The compute path is the C-ABI library ``libtg_gemm.so`` (hand-written CUDA
kernels: TMA, tcgen05.mma into tensor memory, fused ReLU + fp16 epilogue).
This package only marshals arguments to it; the library is loaded on first
use and every call raises if it is missing.
"""
from ._binding import (  # noqa: F401
    A_KM,
    A_MK,
    ACT_GELU,
    ACT_RELU,
    ACT_SILU,
    B_KN,
    B_NK,
    EXPORTS,
    FP8_E4M3,
    FP8_E5M2,
    GatedOptions,
    GemmOptions,
    GroupedOptions,
    LoraOptions,
    LIB_PATH,
    STATIC_WORKSPACE_BYTES,
    Path,
    Status,
    TGError,
    TYPE_BF16,
    TYPE_F16,
    bmm_relu,
    device_status,
    gated_backward_raw,
    gated_backward_workspace_size,
    gated_i8_raw,
    gated_options,
    gated_raw,
    gated_workspace_size,
    gemm_i8_raw,
    grouped_backward_raw,
    grouped_backward_workspace_size,
    grouped_options,
    grouped_raw,
    grouped_workspace_size,
    lora_options,
    lora_raw,
    lora_workspace_size,
    quantize_rows_i8_raw,
    gemm_relu,
    gemm_relu_f16_ex_raw,
    gemm_relu_f16_raw,
    gemm_relu_f16_static_ws_raw,
    gemm_relu_f16_ws_raw,
    gemm_mxf8_grouped_raw,
    gemm_nvf4_grouped_raw,
    gemm_relu_w4a16,
    gemm_relu_w4a16_raw,
    dequant_w4_f16_raw,
    linear_relu,
    lib,
    mx_grouped_rows,
    mx_scale_bytes,
    mxf8_grouped,
    nvf4_grouped,
    nvf4_scale_bytes,
    W4Kernel,
    w4a16_kernel,
    w4a16_workspace_size,
    options,
    path_name,
    path_supports,
    select_path,
    select_path_ex,
    select_path_ws,
    status_string,
    version,
    wait_timeout_selftest,
    workspace_size,
    workspace_size_ex,
)

# The feed-forward operators, the grouped products and the adapters need torch at import; they load with their first use.
_FEEDFORWARD = ("gated", "gated_backward", "gated_block", "gated_i8", "gemm_i8", "quantize_i8")
_EXPERTS = ("grouped", "grouped_backward", "grouped_linear", "lora")


def __getattr__(name):
    if name in _FEEDFORWARD:
        from . import feedforward
        for n in _FEEDFORWARD:
            globals()[n] = getattr(feedforward, n)
        return globals()[name]
    if name in _EXPERTS:
        from . import experts
        for n in _EXPERTS:
            globals()[n] = getattr(experts, n)
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
