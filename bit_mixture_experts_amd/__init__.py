"""moe4: a routed mixture-of-experts expert layer computed directly on 4-bit
expert stacks (NF4 blockwise-absmax or MXFP4), with hand-written HIP kernels for
AMD Instinct MI355X (gfx950); beside it the block's dense operators (residual RMS
norm, MXFP8 quantiser, gated feed-forward block, gradient clipping) and those of a
block held in 4 bits (MXFP4 quantiser, dense MXFP4 product and its input gradient,
the routed layer of a decode step in two launches, the join of two blocks).

The compute path is the C library ``libmoe4.so`` (interface in
``include/moe4.h``); ``bit_mixture_experts_amd.moe4`` is its thin Python
binding. Importing this package does not load the library; importing the
binding does, and fails loudly when the library is missing.
"""

__all__ = ["inputs"]
