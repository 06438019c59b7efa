"""Exact per-row top-K for a DSA sparse-attention indexer on GB300, and the
latent cache and attention around it, and what trains them.

The compute lives in libsatk.so (hand-written sm_103a CUDA kernels behind the
C ABI of include/satk.h); this package only builds it and marshals torch
tensors into it.

    from sparse_attention_indexer_radix_gb300 import topk_rows, dcp_pack, \\
        dcp_topk_pack, dcp_merge_select, dcp_rescue_select, dcp_emit_rows
    from sparse_attention_indexer_radix_gb300 import step_tables, latent_store, \\
        latent_attend, latent_attend_rows, latent_attend_expanded, latent_merge
    from sparse_attention_indexer_radix_gb300 import distill_loss, distill_grad, \\
        latent_rows_weights, latent_attend_expanded_grad
"""
from .binding import (EXPANDED_MAX_QK, EXPANDED_MAX_V, LATENT_MAX, LATENT_MAX_RANKS,
                      LATENT_TAIL_MAX, MERGE_MAX_CANDIDATES, STATUS_BAD_POSITION,
                      STATUS_BAD_REQUEST, STATUS_BAD_ROW, STATUS_DUPLICATE_KEYS,
                      STATUS_NO_BLOCK, STATUS_SLOTS_EXCEEDED, STATUS_STALLED,
                      STATUS_TOO_MANY_TOKENS,
                      TABLES_MAX_REQUESTS, TOPK_MAX_K, SatkError, StepTables, dcp_emit_rows,
                      dcp_merge_select, dcp_pack, dcp_rescue_select, dcp_topk_pack,
                      distill_grad, distill_loss, latent_attend, latent_attend_expanded,
                      latent_attend_expanded_grad, latent_attend_rows,
                      latent_expanded_grad_workspace_bytes, latent_merge, latent_rows_weights,
                      latent_store, latent_workspace_bytes, packed_row_words,
                      rescue_recv_words, rescue_slots, step_tables, topk_rows)

__all__ = ["topk_rows", "dcp_pack", "dcp_topk_pack", "dcp_merge_select", "dcp_rescue_select", "dcp_emit_rows",
           "packed_row_words", "rescue_slots", "rescue_recv_words", "SatkError",
           "STATUS_SLOTS_EXCEEDED", "STATUS_DUPLICATE_KEYS", "STATUS_BAD_REQUEST", "TOPK_MAX_K",
           "MERGE_MAX_CANDIDATES", "step_tables", "StepTables", "latent_store", "latent_attend",
           "latent_attend_rows", "latent_attend_expanded", "latent_merge",
           "latent_workspace_bytes", "STATUS_NO_BLOCK", "STATUS_TOO_MANY_TOKENS",
           "STATUS_BAD_ROW", "STATUS_BAD_POSITION", "STATUS_STALLED", "TABLES_MAX_REQUESTS", "LATENT_MAX",
           "LATENT_TAIL_MAX", "LATENT_MAX_RANKS", "EXPANDED_MAX_QK", "EXPANDED_MAX_V",
           "distill_loss", "distill_grad", "latent_rows_weights", "latent_attend_expanded_grad",
           "latent_expanded_grad_workspace_bytes"]
