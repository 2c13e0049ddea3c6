"""MI355X (gfx950) Kimi Delta Attention chunked operator with a recompute backward.

The operator runs as hand-written HIP kernels behind the C ABI of
``include/kda.h`` (``_build/libkda.so``); this package is its Python binding.
The operators around it in a layer (its recurrent form for decoding) are in
``layer``.
"""
from .ops import (Checkpoints, KDAFunction, KdaError, Problem, kda, kda_backward, kda_forward,
                  kda_forward_noalloc, kda_prologue, gdn2_backward, gdn2_forward)
from .layer import gdn2_recurrent, kda_recurrent

__all__ = ["Checkpoints", "KDAFunction", "KdaError", "Problem", "kda", "kda_backward", "kda_forward",
           "kda_forward_noalloc", "kda_prologue", "gdn2_backward", "gdn2_forward",
           "gdn2_recurrent", "kda_recurrent"]
