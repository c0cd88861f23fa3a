"""MI355X-native MoE expert-layer forward: route -> permute -> grouped GEMM
(gate/up + SwiGLU, down) -> combine, as hand-written HIP kernels for gfx950
behind the C-ABI library ``libmoe.so`` (declared in ``include/moe.h``); beside
it the router's training side (``include/moe_balance.h``), low-rank adapters of
many requests (``include/moe_lora.h``, ``adapters``) and the layer's backward
pass with the clipping of its gradients (``include/moe_backward.h``).

Importing the package does not load the library; ``grouped_gemm_router_amd.api``
does, and raises if it is missing.  ``synth`` holds the seeded input
generators and workload shapes.
"""
__all__ = ["adapters", "api", "layer", "synth"]
