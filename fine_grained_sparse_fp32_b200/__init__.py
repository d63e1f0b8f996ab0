"""Fine-grained sparse MoE feed-forward layer (Kolibri-1 shape) for NVIDIA B200.

The compute path is the CUDA library libkmoe.so (C ABI in include/kmoe.h);
`kmoe` is its thin ctypes binding and `inputs` the seeded input generator.
"""
from . import inputs  # noqa: F401
from .kmoe import (  # noqa: F401
    W4, Experts, KmoeError, Layer, Routing, load, moe_combine, moe_dequant_w4, moe_forward, moe_grouped_ffn,
    moe_linear_w4, moe_permute, moe_quant_w4, moe_route, moe_router_topk, moe_workspace_size, workspace,
)
