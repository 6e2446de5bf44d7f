"""MI355X-native fused clamped-SwiGLU x routing-probability expert activation.

The activation (forward and backward) runs in hand-written HIP kernels for gfx950
behind the C ABI of ``include/swiglu_probs.h``; this package holds the kernels'
sources (``csrc/``), their in-tree build (``build.py``), the ctypes binding
(``swiglu_probs``), the binding of the MoE elementwise operations next to the
activation (``moe_elementwise``: fused residual add, router-weight multiply,
squared-ReLU x probs forward and backward, unpermute in expert order), the binding of the
block's operators around the experts (``moe_block``: layer norm forward and backward, a matrix
product with an epilogue, the router, the expert layer for a few tokens), of the gate behind the
router with its gradient (``moe_gate``) and of the operators on weights in 4 bits (``fp4``), the
HBM probe binding (``hbm_probe``) and the seeded input generators (``workloads``). Libraries are
loaded on first use, not at import.
"""
from .swiglu_probs import (SwigluProbs, SwigluProbsError, backward, forward,  # noqa: F401
                           load_library, swiglu_probs_bwd, swiglu_probs_default_workgroups,
                           swiglu_probs_fwd)

from .moe_elementwise import (FusedMoEResidualAdd, MoeElementwiseError,  # noqa: F401
                              RouterWeightMul, SquaredReluProbs, moe_residual_add,
                              moe_router_weight_bwd, moe_router_weight_fwd,
                              moe_squared_relu_probs_bwd, moe_squared_relu_probs_fwd,
                              moe_unpermute_expert_order)

from .moe_block import (LayerNorm, MoeBlockError, layer_norm_bwd, layer_norm_bwd_workspace,  # noqa: F401
                        layer_norm_fwd, linear_act, linear_act_workspace, moe_experts,
                        moe_experts_workspace, moe_layer, moe_layer_workspace, moe_route,
                        moe_route_workspace)

from .moe_gate import MoeGate, moe_gate_bwd, moe_gate_fwd  # noqa: F401

from .fp4 import (fp4_dequantize, fp4_pack, fp4_quantize, fp4_shapes, linear_act_fp4,  # noqa: F401
                  linear_act_fp4_workspace, moe_experts_fp4, moe_experts_fp4_workspace)

__all__ = ["moe_gate_fwd", "moe_gate_bwd", "MoeGate", "fp4_shapes", "fp4_quantize", "fp4_pack", "fp4_dequantize",
           "linear_act_fp4", "linear_act_fp4_workspace", "moe_experts_fp4", "moe_experts_fp4_workspace",
           "layer_norm_fwd", "layer_norm_bwd", "layer_norm_bwd_workspace", "LayerNorm", "linear_act",
           "linear_act_workspace", "moe_route", "moe_route_workspace", "moe_experts", "moe_experts_workspace",
           "moe_layer", "moe_layer_workspace", "MoeBlockError",
           "moe_residual_add", "moe_router_weight_fwd", "moe_router_weight_bwd",
           "moe_squared_relu_probs_fwd", "moe_squared_relu_probs_bwd", "moe_unpermute_expert_order",
           "FusedMoEResidualAdd", "RouterWeightMul", "SquaredReluProbs", "MoeElementwiseError",
           "swiglu_probs_fwd", "swiglu_probs_bwd", "swiglu_probs_default_workgroups",
           "forward", "backward", "SwigluProbs", "SwigluProbsError", "load_library"]
