"""MXFP8 x MXFP4 fused MoE expert layer for AMD Instinct MI355X (gfx950).

The layer is five C calls into ``libmi355moe.so`` (declared in
``include/mi355moe.h``); this package is their thin Python binding plus
``MoELayer``, which issues the calls in order with one workspace (routing,
quantisation and grouping as the one call ``moe_route_quant_permute``; with
given top-k ids, quantisation and grouping as ``moe_quant_permute``).

Around the experts there are the residual's norm with an 8-bit output, the
router's product, group-limited routing and dense projections in 8-bit
integers; ``MoEBlock`` runs them with a ``MoELayer`` as one MoE block.
"""
from ._binding import (  # noqa: F401
    COMBINE_ATOMIC,
    COMBINE_DETERMINISTIC,
    EXPORTS,
    GROUP_MAX,
    GROUP_TOP2,
    MoEError,
    Q8_INT8,
    Q8_MXFP8,
    Q8_NONE,
    SCORE_SIGMOID,
    SCORE_SOFTMAX,
    lib,
    load_library,
    moe_abi_version,
    moe_add_rmsnorm,
    moe_fc1_situ,
    moe_fc2_combine,
    moe_gate_logits,
    moe_gate_workspace_size,
    moe_int8_linear,
    moe_int8_matmul,
    moe_int8_matmul_workspace_size,
    moe_int8_workspace_size,
    moe_permute,
    moe_permute_noalloc,
    W13_GATE_UP,
    W13_INTERLEAVED,
    W13_UP_GATE,
    moe_prepack_w13,
    moe_prepack_w13_layout,
    moe_prepack_w2,
    moe_quant_int8,
    moe_quant_mxfp8,
    moe_quant_permute,
    moe_route,
    moe_route_groups,
    moe_route_quant_permute,
    moe_workspace_size,
)
from .block import MoEBlock  # noqa: F401
from .layer import MoELayer  # noqa: F401
