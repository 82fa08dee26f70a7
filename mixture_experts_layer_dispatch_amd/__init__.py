"""Single-GPU Mixture-of-Experts layer for AMD Instinct MI355X (gfx950).

The layer (top-k routing, schedule, dispatch, expert-grouped SwiGLU FFN,
weighted combine, and the backward) runs in hand-written HIP kernels behind the
C ABI declared in ``include/moe.h``; this package is the thin Python binding.
"""
from .binding import (Config, LinearConfig, LinearW4Config, MoEError, NormConfig, PREC_BF16, PREC_MXFP8,
                      RouteConfig, alloc_error_word, alloc_grads, alloc_linear_w4_weights,
                      alloc_linear_w4_workspace, alloc_linear_workspace, alloc_norm_workspace, alloc_saved,
                      alloc_schedule,
                      alloc_weights_mx, alloc_workspace, device_supported, lib,
                      linear_w4_workspace_size, linear_workspace_size, moe_backward,
                      moe_check_device_error, moe_forward, moe_linear_backward, moe_linear_forward,
                      moe_linear_w4_forward, moe_linear_w4_quantize, moe_norm_backward, moe_norm_forward,
                      moe_permute_backward, moe_permute_forward, moe_quantize_weights_mxfp8,
                      moe_route_backward, moe_route_forward, moe_schedule, moe_schedule_from_topk,
                      moe_unpermute_backward, moe_unpermute_forward, norm_workspace_size,
                      ring_rows, status_string, validate_config, workspace_size)

__all__ = ["Config", "LinearConfig", "MoEError", "PREC_BF16", "PREC_MXFP8", "alloc_grads", "alloc_saved",
           "alloc_schedule", "alloc_weights_mx", "alloc_workspace", "device_supported", "lib", "moe_backward",
           "moe_check_device_error", "moe_forward", "moe_quantize_weights_mxfp8", "moe_schedule", "ring_rows", "status_string",
           "validate_config", "workspace_size", "alloc_error_word", "alloc_linear_workspace", "linear_workspace_size",
           "moe_linear_backward", "moe_linear_forward", "moe_permute_backward", "moe_permute_forward",
           "moe_unpermute_backward", "moe_unpermute_forward", "LinearW4Config", "NormConfig", "RouteConfig",
           "alloc_linear_w4_weights", "alloc_linear_w4_workspace", "alloc_norm_workspace", "linear_w4_workspace_size",
           "norm_workspace_size", "moe_linear_w4_forward", "moe_linear_w4_quantize", "moe_norm_backward",
           "moe_norm_forward", "moe_route_backward", "moe_route_forward", "moe_schedule_from_topk"]
