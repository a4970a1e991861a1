"""Fused linear cross-entropy for AMD MI355X (gfx950): HIP kernels behind the
C ABI of include/lce.h, with a thin ctypes binding (``lm_head_linear_amd.lce``)."""
from . import lce  # noqa: F401
from .lce import (BeamStep, LceError, LinearGrads, LinearResult, Packed8,  # noqa: F401
                  backward, beam_reorder, beam_select, ce_logits, distill, forward,
                  forward_backward, linear, linear_backward, pack8, unpack8,
                  lce_beam_reorder, lce_beam_select, lce_beam_workspace_bytes, lce_linear,
                  lce_linear_backward, lce_linear_backward_workspace_bytes,
                  lce_linear_workspace_bytes, lce_pack8, lce_unpack8,
                  lce_backward, lce_ce_logits_fwd_bwd, lce_chunk_check, lce_dims_check,
                  lce_distill_fwd_bwd, lce_distill_workspace_bytes, lce_forward,
                  lce_forward_backward, lce_forward_backward_workspace_bytes, lce_logit_cells,
                  lce_loss_fetch,
                  lce_peak_cells, lce_shard_backward, lce_shard_forward, lce_shard_merge,
                  lce_status_name, lce_work_fits, lce_workspace_bytes)
