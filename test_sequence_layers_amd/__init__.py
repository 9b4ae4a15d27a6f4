"""MI355X-native TTT-layer library (HIP kernels for gfx950 behind a C ABI).

The entry points mirror include/ttt.h:
  * forward: ttt_forward_fullbatch, ttt_forward_fullbatch_epochs (several full-batch epochs),
    ttt_forward_chunked_causal, ttt_forward_chunked_bidir, ttt_forward_chunked_bidir2d (raster-
    and column-order bidirectional scans), ttt_mlp_forward;
  * backward (the layers' gradients for the outer loop): ttt_backward_fullbatch,
    ttt_backward_chunked_causal, ttt_backward_chunked_bidir;
  * around the layer: ttt_dwconv3x3 (the depth-wise 3x3 convolution over the token grid that
    precedes a scan or runs beside it), ttt_block_epilogue (ViT^3's gated branch and convolution
    branch concatenated and projected);
  * ttt_forward_fullbatch_noalloc (full-batch with the library's static scratch instead of a
    workspace, for callers that cannot allocate) and ttt_workspace_size.

Those of include/ttt_seq.h, the operators of a block around and beside a TTT layer, each with its
backward pass (seq.py):
  * ttt_forward_layernorm, ttt_backward_layernorm (over a row or per head);
  * ttt_forward_conv1d, ttt_step_conv1d, ttt_backward_conv1d (short causal depth-wise convolution);
  * ttt_forward_selective_scan, ttt_step_selective_scan, ttt_backward_selective_scan (selective state
    space scan); the step forms take one token of every sequence and update its state.

Those of include/ttt_lm.h, the operators of a language model's residual block (lm.py):
  * ttt_forward_rmsnorm, ttt_forward_rmsnorm_e4m3, ttt_backward_rmsnorm (RMS norm with the residual's
    addition, dropout of what is added, and an output in 8 bits);
  * ttt_forward_dropout, ttt_backward_dropout, dropout_counters (dropout whose mask is never stored);
  * ttt_forward_gated_recurrence, ttt_step_gated_recurrence, ttt_backward_gated_recurrence (gated linear
    recurrence, one state per channel).
"""
from .ttt import (  # noqa: F401
    TTT_BF16, TTT_F32, TTT_NOALLOC_SCRATCH_BYTES, TTT_OP_BIDIR, TTT_OP_CAUSAL, TTT_OP_FULLBATCH,
    TTT_OP_BIDIR2D, TTT_OP_BIDIR_BWD, TTT_OP_CAUSAL_BWD, TTT_OP_FULLBATCH_BWD, TTT_OP_MLP,
    TTTError, load_library, status_string, ttt_backward_chunked_bidir, ttt_backward_chunked_causal,
    ttt_backward_fullbatch, ttt_block_epilogue, ttt_forward_chunked_bidir, ttt_forward_chunked_bidir2d, ttt_forward_chunked_causal,
    ttt_dwconv3x3, ttt_forward_fullbatch, ttt_forward_fullbatch_epochs, ttt_forward_fullbatch_noalloc, ttt_mlp_forward, ttt_workspace_size)
from .seq import (  # noqa: F401
    ttt_backward_conv1d, ttt_backward_layernorm, ttt_backward_selective_scan, ttt_forward_conv1d, ttt_forward_layernorm,
    ttt_forward_selective_scan, ttt_step_conv1d, ttt_step_selective_scan)
from .lm import (  # noqa: F401
    dropout_counters, ttt_backward_dropout, ttt_backward_gated_recurrence, ttt_backward_rmsnorm, ttt_forward_dropout,
    ttt_forward_gated_recurrence, ttt_forward_rmsnorm, ttt_forward_rmsnorm_e4m3, ttt_step_gated_recurrence)
