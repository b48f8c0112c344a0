"""MI355X-native MoE decode layer (DeepSeek-V4.1-Flash style): Q2_K/Q3_K
routed experts on raw blocks, bf16 router and shared expert.

The compute lives in libmoe.so (hand-written HIP for gfx950, C ABI declared
in include/moe.h); this package only marshals arguments to it.
"""
from .binding import (MOE_K_DOWN, MOE_K_DOWN2, MOE_K_GATEUP, MOE_K_GATEUP2, MOE_K_READ_PROBE, MOE_K_ROUTER, MOE_K_SHARED_DOWN, MOE_K_SHARED_GU,
                      MOE_SCORE_CR, MOE_SCORE_GLIBC, MOE_SHARED_BF16, MOE_SHARED_KQUANT,
                      MOE_STATUS_BAD_PICK, MOE_STATUS_MISS, MOE_STATUS_NAN_KEY, SCORES_EXP_ONLY, SCORES_EXTENDED, SCORES_GLIBC, Cfg, ExpertCache, Experts, Layer, MoeError,
                      cfg_from_shape, enable_glibc_scores, experts_decode, glibc_score_table, experts_prefill, header_words, layer_forward, layer_forward_noalloc, lib, read_probe,
                      lru_simulate, route_select, scores, scores_host, stack_forward, swiglu_host, time_next_launch,
                      workspace_bytes, workspace_init, workspace_layout)
from .binding import (MOE_ADAPTER_MAX_ADAPTERS, MOE_ADAPTER_MAX_RANK, MOE_ADAPTER_MAX_TOKENS, MOE_GROUPED_MAX_GROUPS, MOE_GROUPED_MAX_ROWS, MOE_GROUPED_MAX_STRIDE, MOE_JOIN_MAX_DIM, MOE_STATUS_BAD_ADAPTER, MOE_STATUS_BAD_OFFSETS, MOE_TYPE_BF16, MOE_TYPE_F32,
                      MOE_TYPE_FP16, Adapters, Grouped, Join,
                      MOE_MX_CEIL, MOE_MX_FLOOR, MOE_MX_MAX_K, MOE_MX_MAX_ROWS, Mx, MxRows, mx_dequantise, mx_forward, mx_gated, mx_quantise,
                      MOE_ACT_GELU, MOE_ACT_SILU, Gated, act_code, gated_backward_h, gated_backward_x, gated_forward,
                      adapter_project, adapter_workspace_bytes, grouped_backward_w, grouped_backward_x, grouped_forward, join_backward, join_forward, join_workspace_bytes, type_code)

__all__ = [
    "Cfg", "ExpertCache", "Experts", "Layer", "MoeError", "cfg_from_shape", "enable_glibc_scores", "experts_decode",
    "glibc_score_table", "experts_prefill", "header_words",
    "layer_forward", "layer_forward_noalloc", "lib", "lru_simulate", "read_probe", "route_select", "scores", "scores_host", "stack_forward", "swiglu_host",
    "time_next_launch", "workspace_bytes", "workspace_init", "workspace_layout", "MOE_K_GATEUP", "MOE_K_DOWN",
    "MOE_K_ROUTER", "MOE_K_READ_PROBE", "MOE_K_SHARED_GU", "MOE_K_SHARED_DOWN", "MOE_K_GATEUP2", "MOE_K_DOWN2",
    "MOE_SCORE_CR", "MOE_SCORE_GLIBC", "MOE_SHARED_BF16", "MOE_SHARED_KQUANT", "MOE_STATUS_MISS", "MOE_STATUS_NAN_KEY", "MOE_STATUS_BAD_PICK", "SCORES_EXTENDED", "SCORES_GLIBC", "SCORES_EXP_ONLY",
    "Join", "join_backward", "join_forward", "join_workspace_bytes", "type_code", "MOE_TYPE_BF16", "MOE_TYPE_FP16",
    "MOE_TYPE_F32", "MOE_STATUS_BAD_OFFSETS", "MOE_STATUS_BAD_ADAPTER", "MOE_JOIN_MAX_DIM",
    "Grouped", "grouped_forward", "grouped_backward_x", "grouped_backward_w", "MOE_GROUPED_MAX_GROUPS",
    "MOE_GROUPED_MAX_ROWS", "MOE_GROUPED_MAX_STRIDE", "Adapters", "adapter_project", "adapter_workspace_bytes", "MOE_ADAPTER_MAX_ADAPTERS",
    "MOE_ADAPTER_MAX_RANK", "MOE_ADAPTER_MAX_TOKENS",
    "Gated", "act_code", "gated_forward", "gated_backward_h", "gated_backward_x", "MOE_ACT_SILU", "MOE_ACT_GELU",
    "MxRows", "mx_quantise", "mx_dequantise", "Mx", "mx_forward", "mx_gated", "MOE_MX_FLOOR", "MOE_MX_CEIL", "MOE_MX_MAX_K",
    "MOE_MX_MAX_ROWS",
]
