"""Grouped 4-bit mixture-of-experts GEMM for AMD MI355X (gfx950).

The compute path is the HIP library libgnf4.so (csrc/, C ABI in
include/gnf4.h); ``gnf4`` is its Python binding. Build with
``python -m bit_mixture_experts_topk_amd.build``.
"""

from . import gnf4  # noqa: F401
from .gnf4 import (KVBatch, KVCache, MXFP4, NF4, NF4_DQ, PackedWeights, Rope, build_id, combine,  # noqa: F401
                   dequant, empty_kv_cache, grouped_gemm, kv_attention, kv_cache_read, kv_cache_write,
                   qk_norm_rope, qk_norm_rope_dx, quantize, rope_frequencies, route)
