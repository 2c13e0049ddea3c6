"""MI355X (gfx950) Kimi Delta Attention chunked operator with a recompute backward.

The operator runs as hand-written HIP kernels behind the C ABI of
``include/kda.h`` (``_build/libkda.so``); this package is its Python binding.
The operators around it in a layer (the short convolution in front of it, its
recurrent form for decoding, the norm behind it with the output gate, the norms
between blocks) are in ``layer``, those of a state-space layer (the selective
scan, its decoding form, group norm) in ``ssm``.
"""
from .ops import (Checkpoints, KDAFunction, KdaError, Problem, kda, kda_backward, kda_forward,
                  kda_forward_noalloc, kda_prologue, gdn2_backward, gdn2_forward)
from .layer import (BlockNormFunction, GatedNormFunction, ShortConvFunction, block_norm,
                    block_norm_backward, block_norm_forward, gated_norm, gated_norm_backward,
                    gated_norm_forward, gdn2_recurrent, kda_recurrent, short_conv,
                    short_conv_backward, short_conv_forward, short_conv_update)
from .ssm import (GroupNormFunction, SsmScanFunction, group_norm, group_norm_backward,
                  group_norm_forward, ssm_recurrent, ssm_scan, ssm_scan_backward, ssm_scan_forward)

__all__ = ["Checkpoints", "KDAFunction", "KdaError", "Problem", "kda", "kda_backward", "kda_forward",
           "kda_forward_noalloc", "kda_prologue", "gdn2_backward", "gdn2_forward",
           "gdn2_recurrent", "kda_recurrent", "GatedNormFunction", "gated_norm",
           "gated_norm_forward", "gated_norm_backward", "BlockNormFunction", "block_norm",
           "block_norm_forward", "block_norm_backward", "ShortConvFunction", "short_conv",
           "short_conv_forward", "short_conv_backward", "short_conv_update", "SsmScanFunction",
           "ssm_scan", "ssm_scan_forward", "ssm_scan_backward", "ssm_recurrent",
           "GroupNormFunction", "group_norm", "group_norm_forward", "group_norm_backward"]
