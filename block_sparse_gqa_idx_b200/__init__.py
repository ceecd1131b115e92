"""MiniMax Sparse Attention (MSA) forward path for B200 (sm_100a).

The compute lives in ``libmsa_b200.so`` (hand-written CUDA behind the C ABI
of ``include/msa.h``); this package is its thin Python binding:

* ``index_topk``      Index Branch, Eq. 6-7 (fused scores, block max, Top-k)
* ``sparse_attn_fwd`` Main Branch, Eq. 8 (KV-outer sparse attention + merge)
* ``forward``         both, for one prefill sequence
* ``forward_varlen``  both, for a packed batch of sequences of any lengths
* ``project``         the Q, K, V and index projections upstream of the path
* ``sparse_attn_bwd`` the backward of the Main Branch (dQ, dK, dV)
* ``sparse_decode``   one decode step for a batch of sequences
* ``paged_decode_fp8`` the same step on a paged FP8 (E4M3) KV cache
* ``qk_norm_rope``    per-head RMS norm + position rotation of q and k (and
  ``qk_norm_rope_bwd``), between the projections and the attention
* ``paged_append_fp8``, ``paged_gather_fp8``  a chunk of new tokens quantised
  into the paged FP8 cache, and cached tokens read back (``chunk_positions``:
  the positions of a chunk's rows)
* ``paged_index_scores_fp8``, ``block_topk``  the Index Branch of a chunk on
  that cache: block scores, and the selection from them
* ``paged_sparse_attn_fp8``  the Main Branch of a chunk on that cache
* ``paged_chunk_fp8``  the whole step for a chunk: append, selection, attention

``inputs`` holds the seeded synthetic workload generators.  The binding is
loaded on first use of one of the names above and raises if the CUDA library
has not been built (``python -m block_sparse_gqa_idx_b200.build``).
"""
_CAPI = ("index_topk", "sparse_attn_fwd", "forward", "sparse_decode", "device_status",
         "version", "MSAError", "dims", "decode_dims", "index_topk_workspace_size",
         "sparse_attn_fwd_workspace_size", "sparse_decode_workspace_size", "EXPORTS", "LIB_PATH",
         "profile_enable", "profile_read", "sparse_decode_noalloc", "selftest_bounded_wait",
         "index_lse", "index_lse_workspace_size", "paged_dims", "paged_decode_fp8",
         "paged_decode_fp8_workspace_size", "quantize_fp8_rows", "index_topk_varlen",
         "sparse_attn_fwd_varlen", "forward_varlen", "varlen_dims", "project",
         "varlen_workspace_size", "sparse_attn_bwd",
         "sparse_attn_bwd_workspace_size", "qk_norm_rope", "qk_norm_rope_bwd",
         "chunk_dims", "chunk_positions", "paged_append_fp8", "paged_gather_fp8",
         "paged_index_scores_fp8", "block_topk", "paged_sparse_attn_fp8",
         "paged_sparse_attn_fp8_workspace_size", "paged_chunk_fp8", "paged_chunk_fp8_workspace_size")

__all__ = list(_CAPI) + ["inputs"]


def __getattr__(name):
    if name in _CAPI:
        from . import _capi

        value = globals()[name] = getattr(_capi, name)  # found directly from now on
        return value
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
