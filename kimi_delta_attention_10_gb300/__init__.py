"""GB300 (sm_103a) chunked Kimi Delta Attention forward and backward.

The compute path is libkda_gb300.so (C ABI in include/kda.h), reached through
``kda_gate``, ``kda_chunk_fwd``, ``kda_chunk_fwd_gated`` and
``kda_recurrent_step`` (``chunk_workspace_size`` sizes the two-phase path's
scratch; ``kda_chunk_fwd_static`` runs it on the library's own scratch),
``kda_gated_rmsnorm`` (the output gate; ``kda_chunk_fwd_gated_norm`` fuses it
into the forward) and ``kda_chunk_bwd`` (the VJP,
scratch sized by ``chunk_bwd_workspace_size``).  Full attention beside the KDA
layers is served by ``kda_page_plan`` (block tables and slots from lengths),
``kda_qk_norm_rope`` with its backward ``kda_qk_norm_rope_bwd`` and its
cache-writing form ``kda_qk_norm_rope_append`` (``rope_inv_freq`` makes the
frequencies) and ``kda_paged_decode`` (one new token over the pages);
``inputs`` holds the seeded synthetic workloads.
"""
from .binding import (KDAError, chunk_bwd_workspace_size, chunk_workspace_size,  # noqa: F401
                      kda_chunk_bwd, kda_chunk_fwd, kda_chunk_fwd_gated, kda_chunk_fwd_gated_norm,
                      kda_chunk_fwd_static,
                      kda_gate, kda_gated_rmsnorm, kda_page_plan, kda_paged_decode,
                      kda_qk_norm_rope, kda_qk_norm_rope_append, kda_qk_norm_rope_bwd,
                      kda_recurrent_step, library_path, load_library,
                      paged_decode_workspace_size, qk_norm_rope_bwd_workspace_size,
                      rope_inv_freq, status_string)
