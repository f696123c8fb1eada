"""GB300 (sm_103a) three-tier compressed attention of the DeepSeek V4 Flash
engine (DwarfStar, ds4): indexer score -> top-k select -> sparse attention,
hand-written CUDA behind the C ABI of include/ds4a.h.

The Python surface is the ctypes binding (same names as the C entry points)
and DecodeStep / PrefillStep, which chain the three ops on one stream, plus
DenseStep for the ratio-128 layers (attention over all rows, no indexer) and
PagedDecodeStep, a decode step over caches in pages (lengths -> block tables and
slots -> norm and rotation -> score -> select -> attention).
"""
from ._binding import (Ds4aError, load, ds4a_version, ds4a_workspace_bytes, ds4a_get_device_status,
                       ds4a_debug_inject_error, ds4a_debug_wait_timeout, ds4a_indexer_score, ds4a_topk_select,
                       ds4a_sparse_attn_decode, ds4a_sparse_attn_prefill, ds4a_dense_attn_decode,
                       ds4a_kv_push_raw, ds4a_compressor_pool, ds4a_sparse_attn_decode_heads,
                       ds4a_sparse_attn_prefill_heads, ds4a_dense_attn_decode_heads, ds4a_rows_to_fp8,
                       ds4a_sparse_attn_decode_fp8, ds4a_sparse_attn_prefill_fp8, ds4a_indexer_topk,
                       ds4a_paged_plan, ds4a_qk_norm_rope, ds4a_paged_indexer_score, ds4a_paged_attn_decode,
                       DS4A_OP_PAGED_ATTN_DECODE, DS4A_PLAN_TOKENS_BY_SEQ, DS4A_PLAN_ROWS_BY_SEQ, DS4A_PLAN_FIRST_POS,
                       DS4A_OP_FLAG_128_HEADS, DS4A_ROPE_NEIGHBOURS, DS4A_ROPE_HALVES)
from .step import DecodeStep, PrefillStep, DenseStep, ProducerStep, PagedDecodeStep, DEFAULT_SCALE

__all__ = ["Ds4aError", "load", "ds4a_version", "ds4a_workspace_bytes", "ds4a_get_device_status",
           "ds4a_debug_inject_error", "ds4a_debug_wait_timeout", "ds4a_indexer_score", "ds4a_topk_select", "ds4a_sparse_attn_decode",
           "ds4a_sparse_attn_prefill", "ds4a_dense_attn_decode", "ds4a_kv_push_raw", "ds4a_compressor_pool",
           "ds4a_sparse_attn_decode_heads", "ds4a_sparse_attn_prefill_heads", "ds4a_dense_attn_decode_heads",
           "ds4a_rows_to_fp8", "ds4a_sparse_attn_decode_fp8", "ds4a_sparse_attn_prefill_fp8", "ds4a_indexer_topk",
           "ds4a_paged_plan", "ds4a_qk_norm_rope", "ds4a_paged_indexer_score", "ds4a_paged_attn_decode",
           "DS4A_OP_PAGED_ATTN_DECODE", "DS4A_PLAN_TOKENS_BY_SEQ", "DS4A_PLAN_ROWS_BY_SEQ", "DS4A_PLAN_FIRST_POS",
           "DS4A_OP_FLAG_128_HEADS", "DS4A_ROPE_NEIGHBOURS", "DS4A_ROPE_HALVES",
           "DecodeStep", "PrefillStep", "DenseStep", "ProducerStep", "PagedDecodeStep",
           "DEFAULT_SCALE"]
