"""GB300 (sm_103a) SwiGLU FFN and top-k MoE forward behind a C ABI (libmm.so).

Public API: swiglu_ffn, moe_forward, moe_route, check_status (see api.py),
and what surrounds the experts' products with its gradients: block norms,
tokens sorted by expert, 8-bit activation checkpoints (see block_ops.py), and
the experts' products, in bf16, fp32 or 4-bit floating point (see products.py);
the C entry points are declared in include/mm.h.
"""
from .api import (  # noqa: F401
    swiglu_ffn_backward, moe_backward, swiglu_block, prepare_down_weights,
    swiglu_ffn, swiglu_ffn_noalloc, moe_forward, moe_route, check_status, watchdog_selftest,
    ffn_workspace_bytes, moe_workspace_bytes, new_workspace,
)
from .block_ops import (  # noqa: F401
    block_norm, block_norm_backward, block_norm_backward_workspace_bytes,
    moe_permute, moe_permute_backward, moe_permute_workspace_bytes, moe_permuted_rows,
    moe_unpermute, moe_unpermute_backward,
    checkpoint_pack, checkpoint_unpack, swiglu_act, swiglu_act_backward,
)
from .products import (  # noqa: F401
    grouped_matmul, grouped_matmul_backward, grouped_matmul_backward_workspace_bytes,
    grouped_matmul_workspace_bytes, mx4_dequantize, mx4_matmul, mx4_matmul_workspace_bytes, mx4_quantize,
)
