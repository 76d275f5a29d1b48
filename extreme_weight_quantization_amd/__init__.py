"""AQLM 2-bit quantized linear layer for AMD Instinct MI355X (gfx950).

The compute path is a C-ABI shared library of hand-written HIP kernels
(``libaqlm.so``, declared in ``include/aqlm.h``).  ``binding`` is the thin
ctypes layer over it, ``fused`` that of the products with an epilogue, the gated
product and their backward passes; ``synth`` draws seeded synthetic layers.  The library
is loaded on first use and its absence is an error: there is no fallback.
"""
from .binding import (  # noqa: F401
    AqlmError,
    SliceLists,
    aqlm_linear_gemv_lists,
    aqlm_linear_gemv_lists_fused,
    aqlm_linear_gemv_lists_noalloc,
    aqlm_pack_codes,
    aqlm_linear_gemv_packed,
    aqlm_linear_gemm_packed,
    aqlm_linear_decode_packed,
    packed_codes_bytes,
    aqlm_lists_pack,
    aqlm_linear_decode,
    aqlm_linear_gemm,
    aqlm_linear_gemm_dequant,
    gemm_dequant_workspace_bytes,
    aqlm_linear_gemv,
    aqlm_linear_gemv_fused,
    aqlm_encode_greedy,
    aqlm_kmeans_init,
    kmeans_workspace_bytes,
    lists_fused_workspace_bytes,
    lists_table_bytes,
    lists_workspace_bytes,
    load_library,
    status_str,
)
from .fused import (  # noqa: F401
    ACTIVATIONS,
    aqlm_gated,
    aqlm_gated_backward,
    aqlm_gated_lists,
    aqlm_linear_act,
    aqlm_linear_act_backward,
    aqlm_linear_act_lists,
    gated_backward_workspace_bytes,
    gated_workspace_bytes,
    linear_act_backward_workspace_bytes,
    linear_act_workspace_bytes,
)
from .moe import (  # noqa: F401
    SCORES,
    aqlm_moe,
    aqlm_moe_mx4,
    aqlm_moe_route,
    moe_mx4_workspace_bytes,
    moe_route_workspace_bytes,
    moe_workspace_bytes,
)
from .mx4 import (  # noqa: F401
    aqlm_mx4_decode,
    aqlm_mx4_linear,
    aqlm_mx4_quantize,
    mx4_linear_workspace_bytes,
)
