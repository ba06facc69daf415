"""MI355X-native routed MoE expert layer with fused rank-r side-LoRA.

The hot path is hand-written HIP for gfx950 behind the C ABI in
include/moelora.h (libmoelora.so, built in-tree by ``build.py``).  Around it
stand the router (``MoeRouter``), the optimiser step of the adapter factors
(``MoeAdamW``) and the expert products in 8-bit floating point
(``fp8_quantize_rows``, ``fp8_quantize_weight``, ``fp8_product``).  This
package adds the ctypes binding (``binding``), the build script and the seeded
synthetic inputs (``inputs``).
"""
from .binding import (  # noqa: F401
    MoeAdamW, MoeLoraDesc, MoeLoraError, MoeLoraLayer, MoeRouter, build_pool, fp8_product, fp8_quantize_rows,
    fp8_quantize_weight, library, make_desc, moe_lora_backward,
    moe_lora_block_m, moe_lora_forward, moe_lora_pool_capacity, moe_lora_workspace_size,
)
