"""Segmented MXFP8 GEMM for AMD Instinct MI355X (gfx950).

The compute half of a fused all-to-all + MXFP8 matmul: R simulated ranks'
A segments are staged chunk by chunk into a ring of buffers and consumed by
a block-scaled FP8 GEMM on CDNA4 scaled MFMA, producing bfloat16 C.  The
work runs in the HIP library ``libmxgemm_seg.so`` behind the C ABI in
``include/mxgemm_seg.h``; this package is its thin Python binding.  The expert
layer around the product (tokens sorted by expert, dispatched and combined;
MXFP8 products with a fused epilogue; their gradients) is in the same library,
behind ``include/mxgemm_moe.h``.
"""
from ._lib import (  # noqa: F401
    EXPORTED, FMT_E4M3, FMT_E5M2, PRECISION_EXACT, PRECISION_NATIVE, RING_EVENTS, RING_FLAGS,
    MxgemmError, Options, Plan, SegGemm, decode,
    last_error, load, options, plan, quantize_mxfp8, quantize_segments, run_static,
)
from ._moe import (  # noqa: F401
    EXPORTED_MOE, LinearGrads, TokenSort, combine_tokens, combine_tokens_backward, dispatch_tokens,
    dispatch_tokens_backward, dispatch_tokens_mx, epilogue_backward, linear, linear_backward, linear_by_inner,
    quantize_transposed, sort_tokens,
)
