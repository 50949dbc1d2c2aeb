"""FP8 W8A8 block-scaled linear layers for AMD MI355X (gfx950).

The computation lives in libfp8w8a8.so (hand-written HIP kernels behind a C
ABI declared in include/fp8w8a8.h, for the paged attention step in
include/fp8w8a8_attention.h and for what runs around both in
include/fp8w8a8_step.h); this package is its Python binding.
"""

from ._attention import (  # noqa: F401
    attention_workspace_bytes, kv_slot_map, paged_attention, prefix_attention, qk_norm_rope_cache,
)
from ._lib import (  # noqa: F401
    LIB_PATH, SCALE_BLOCK, SCALE_ROW, SCALE_TENSOR, block_gemm, encode_f32, grouped_gemm,
    kv_cache_read, kv_cache_write, lib, linear, linear_noalloc, quant_act, quant_act_static, quant_weight_block,
    status_str, workspace_bytes,
)
from ._step import (  # noqa: F401
    MAX_TOP, add_rms_norm, add_rms_norm_quant, int4_linear, int4_pack, int4_quant_weight,
    int4_workspace_bytes, logprobs_workspace_bytes, qk_norm_mrope_cache, token_logprobs,
)
