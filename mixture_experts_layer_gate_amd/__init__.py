"""MI355X (gfx950) DeepSeekMoE layer forward: HIP kernels behind a C ABI.

``binding`` mirrors include/moe.h call for call; ``layer.MoELayer`` composes
the five calls into one layer forward plus the step-end bias update;
``attention.PrefixAttention`` composes the cache append and the attention of a
decode batch that shares a prompt, ``attention.AttentionLayer`` the norm, the
rotary positions and the causal attention of training sequences, both ways.
"""
from . import binding  # noqa: F401
from .binding import (  # noqa: F401
    MoEError, moe_shape, moe_route, moe_permute, moe_grouped_ffn, moe_combine, moe_bias_update,
    moe_quantize_weights, moe_workspace_bytes, moe_ffn_gate_up, moe_ffn_down, MOE_F32, MOE_BF16, MOE_F8E4M3, MOE_ROWS_DIRECT,
    MOE_ROWS_GATHER, MOE_ROWS_SEGMENT, MOE_ROPE_HALF, MOE_ROPE_INTERLEAVED, MOE_ROPE_PLAIN, MOE_ROPE_LINEAR,
    MOE_ROPE_BASE, MOE_ROPE_PARTS, moe_rope_table, moe_rotary, moe_rotary_backward, moe_kv_append,
    moe_prefix_attention, moe_prefix_attention_workspace_bytes, moe_causal_attention, moe_causal_attention_backward,
    moe_causal_attention_backward_workspace_bytes, moe_layer_norm, moe_layer_norm_backward,
    moe_layer_norm_backward_workspace_bytes,
)
from .layer import MoELayer, StepGraph  # noqa: F401
from .attention import AttentionLayer, PrefixAttention  # noqa: F401
