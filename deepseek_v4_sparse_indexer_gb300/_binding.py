"""ctypes binding of libds4a.so: the C ABI's entry points under the same names.

Argument marshalling only: each function checks dtypes, shapes, devices and
contiguity of torch tensors, passes their device pointers, the sizes and the
current CUDA stream to the C entry point, and raises Ds4aError on a non-zero
status.  Every step of the computation runs in the library's CUDA kernels;
there is no CPU path.  If the shared library is missing or cannot be loaded,
load() raises: nothing falls back.
"""
import ctypes
import os

import torch

from . import build as _build

DS4A_OK = 0
DS4A_EINVAL = -1
DS4A_EUNSUPPORTED = -2
DS4A_ECUDA = -3
DS4A_EWORKSPACE = -4
DS4A_EDEVICE = -5
DS4A_DEV_TIMEOUT = 1
DS4A_DEV_BOUNDS = 2
DS4A_OP_INDEXER_SCORE = 0
DS4A_OP_TOPK_SELECT = 1
DS4A_OP_SPARSE_ATTN_DECODE = 2
DS4A_OP_SPARSE_ATTN_PREFILL = 3
DS4A_OP_DENSE_ATTN_DECODE = 4
DS4A_OP_INDEXER_TOPK = 5
DS4A_OP_PAGED_ATTN_DECODE = 6
DS4A_OP_PAGED_ATTN_BLOCKS = 7
DS4A_OP_PAGED_EVICT = 8
DS4A_OP_FLAG_128_HEADS = 0x100
DS4A_BF16, DS4A_F16, DS4A_F32, DS4A_E4M3 = 0, 1, 2, 3
DS4A_ROPE_NEIGHBOURS, DS4A_ROPE_HALVES = 0, 1
DS4A_LIST_ROWS, DS4A_LIST_BLOCKS = 0, 1
DS4A_SCALE_POW2, DS4A_SCALE_MAX = 0, 1
DS4A_MAX_NORM_DIM = 16384
DS4A_MIN_PAGE, DS4A_MAX_PAGE, DS4A_MAX_PLAN_SEQS = 8, 4096, 8192
DS4A_PLAN_TOKENS_BY_SEQ, DS4A_PLAN_ROWS_BY_SEQ, DS4A_PLAN_FIRST_POS = 1, 2, 4

N_HEAD, HEAD_DIM, N_IDX_HEAD, IDX_DIM, N_SWA = 64, 512, 64, 128, 128

# The C entry points this binding (and include/ds4a.h) exposes.
EXPORTS = ("ds4a_strerror", "ds4a_version", "ds4a_workspace_bytes", "ds4a_get_device_status",
           "ds4a_debug_inject_error", "ds4a_debug_wait_timeout", "ds4a_indexer_score", "ds4a_topk_select",
           "ds4a_topk_select_noalloc", "ds4a_sparse_attn_decode", "ds4a_sparse_attn_prefill",
           "ds4a_dense_attn_decode", "ds4a_kv_push_raw", "ds4a_compressor_pool",
           "ds4a_sparse_attn_decode_heads", "ds4a_sparse_attn_prefill_heads", "ds4a_dense_attn_decode_heads",
           "ds4a_rows_to_fp8", "ds4a_sparse_attn_decode_fp8", "ds4a_sparse_attn_prefill_fp8", "ds4a_indexer_topk",
           "ds4a_paged_plan", "ds4a_paged_plan_form", "ds4a_qk_norm_rope", "ds4a_paged_indexer_score",
           "ds4a_paged_attn_decode", "ds4a_paged_block_keys", "ds4a_paged_block_score", "ds4a_paged_attn_blocks",
           "ds4a_paged_attn_mass", "ds4a_paged_evict", "ds4a_paged_evict_shared", "ds4a_add_rms_norm", "ds4a_paged_plan_evicted")
DS4A_TOPK_NOALLOC_SCRATCH_BYTES = 8 << 20
DS4A_MAX_TOP_K = 2048


class Ds4aError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: ds4a status {status} ({_strerror(status)})")


_lib = None
_vp, _i32, _i64, _f32, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


def lib_path() -> str:
    return _build.LIB_PATH


def load(build_if_missing: bool = True):
    """Load libds4a.so (building it with nvcc first if it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB_PATH
    if build_if_missing and not _build.up_to_date():
        _build.build()
    if not os.path.exists(path):
        raise RuntimeError(f"libds4a.so not found at {path}; build it with __graft_entry__.build()")
    L = ctypes.CDLL(path)
    L.ds4a_strerror.argtypes = [_i32]
    L.ds4a_strerror.restype = ctypes.c_char_p
    L.ds4a_version.restype = _i32
    L.ds4a_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32, _i32]
    L.ds4a_workspace_bytes.restype = _sz
    L.ds4a_get_device_status.argtypes = [_vp, ctypes.POINTER(ctypes.c_uint)]
    L.ds4a_get_device_status.restype = _i32
    L.ds4a_debug_inject_error.argtypes = [_i32]
    L.ds4a_debug_inject_error.restype = None
    L.ds4a_debug_wait_timeout.argtypes = [ctypes.c_uint, _vp]
    L.ds4a_debug_wait_timeout.restype = _i32
    L.ds4a_indexer_score.argtypes = [_vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp]
    L.ds4a_indexer_score.restype = _i32
    L.ds4a_topk_select.argtypes = [_vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _sz, _vp]
    L.ds4a_topk_select.restype = _i32
    L.ds4a_topk_select_noalloc.argtypes = [_vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp]
    L.ds4a_topk_select_noalloc.restype = _i32
    L.ds4a_sparse_attn_decode.argtypes = [_vp, _vp, _i64, _i32, _vp, _vp, _i32, _vp, _i64, _vp, _f32, _vp, _vp,
                                          _i32, _vp, _sz, _vp]
    L.ds4a_dense_attn_decode.argtypes = [_vp, _vp, _i64, _i32, _vp, _vp, _i64, _vp, _f32, _vp, _vp, _i32, _vp, _sz,
                                         _vp]
    L.ds4a_dense_attn_decode.restype = _i32
    L.ds4a_kv_push_raw.argtypes = [_vp, _vp, _i64, _vp, _vp, _i32, _vp]
    L.ds4a_kv_push_raw.restype = _i32
    L.ds4a_compressor_pool.argtypes = [_vp, _vp, _i32, _i32, _vp, _i32, _vp]
    L.ds4a_compressor_pool.restype = _i32
    L.ds4a_sparse_attn_decode.restype = _i32
    L.ds4a_sparse_attn_prefill.argtypes = [_vp, _vp, _vp, _i32, _vp, _vp, _i32, _vp, _i32, _i32, _f32, _vp, _vp,
                                           _i32, _vp, _sz, _vp]
    L.ds4a_sparse_attn_prefill.restype = _i32
    L.ds4a_sparse_attn_decode_heads.argtypes = [_i32] + L.ds4a_sparse_attn_decode.argtypes
    L.ds4a_sparse_attn_decode_heads.restype = _i32
    L.ds4a_sparse_attn_prefill_heads.argtypes = [_i32] + L.ds4a_sparse_attn_prefill.argtypes
    L.ds4a_sparse_attn_prefill_heads.restype = _i32
    L.ds4a_dense_attn_decode_heads.argtypes = [_i32] + L.ds4a_dense_attn_decode.argtypes
    L.ds4a_dense_attn_decode_heads.restype = _i32
    L.ds4a_indexer_topk.argtypes = [_vp, _vp, _vp, _i64, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _sz,
                                    _vp]
    L.ds4a_indexer_topk.restype = _i32
    L.ds4a_rows_to_fp8.argtypes = [_vp, _i64, _vp, _vp, _vp]
    L.ds4a_rows_to_fp8.restype = _i32
    L.ds4a_sparse_attn_decode_fp8.argtypes = [_vp, _vp, _vp, _i64, _i32, _vp, _vp, _i32, _vp, _i64, _vp, _f32, _vp,
                                              _vp, _i32, _vp, _sz, _vp]
    L.ds4a_sparse_attn_decode_fp8.restype = _i32
    L.ds4a_sparse_attn_prefill_fp8.argtypes = [_vp, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _vp, _i32, _i32, _f32, _vp,
                                               _vp, _i32, _vp, _sz, _vp]
    L.ds4a_sparse_attn_prefill_fp8.restype = _i32
    L.ds4a_paged_plan.argtypes = [_vp, _vp, _i32, _i32, _i32, _vp, _i32, _vp, _vp, _vp, _i64, _i32, _vp, _vp, _vp, _vp,
                                  _vp, _vp, _vp, _i32, _vp, _vp, _i32, _vp]
    L.ds4a_paged_plan.restype = _i32
    L.ds4a_paged_plan_form.argtypes = [_i32] + L.ds4a_paged_plan.argtypes
    L.ds4a_paged_plan_form.restype = _i32
    L.ds4a_paged_plan_evicted.argtypes = [_i32, _vp, _vp] + L.ds4a_paged_plan.argtypes[1:]
    L.ds4a_paged_plan_evicted.restype = _i32
    L.ds4a_qk_norm_rope.argtypes = [_vp, _i32, _i64, _vp, _i32, _i64, _vp, _vp, _i32, _i32, _f32, _vp, _vp, _vp, _vp,
                                    _i32, _vp, _vp, _i64, _i32, _i32, _i32, _vp]
    L.ds4a_qk_norm_rope.restype = _i32
    L.ds4a_paged_indexer_score.argtypes = [_vp, _vp, _vp, _i32, _i32, _vp, _i64, _i32, _vp, _vp, _i32, _i32, _vp]
    L.ds4a_paged_indexer_score.restype = _i32
    L.ds4a_paged_attn_decode.argtypes = [_i32, _vp, _vp, _i32, _vp, _i32, _i32, _vp, _i64, _i32, _vp, _vp, _vp, _i32,
                                         _vp, _i32, _vp, _vp, _f32, _vp, _vp, _i32, _vp, _sz, _vp]
    L.ds4a_paged_attn_decode.restype = _i32
    L.ds4a_paged_block_keys.argtypes = [_vp, _i32, _i32, _vp, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _i32, _vp]
    L.ds4a_paged_block_keys.restype = _i32
    L.ds4a_paged_block_score.argtypes = [_vp, _vp, _vp, _i32, _vp, _i64, _i32, _vp, _i32, _i32, _vp, _i32, _i32, _vp]
    L.ds4a_paged_block_score.restype = _i32
    L.ds4a_paged_attn_blocks.argtypes = L.ds4a_paged_attn_decode.argtypes
    L.ds4a_paged_attn_blocks.restype = _i32
    L.ds4a_paged_attn_mass.argtypes = [_i32, _vp, _vp, _i32, _vp, _i32, _i32, _vp, _i64, _i32, _vp, _i32, _vp, _vp, _i32,
                                       _f32, _vp, _vp, _vp, _i64, _i32, _vp]
    L.ds4a_paged_attn_mass.restype = _i32
    L.ds4a_paged_evict.argtypes = [_vp, _i32, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i32, _i32, _i32,
                                   _i32, _i32, _vp, _i32, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                   _sz, _vp]
    L.ds4a_paged_evict.restype = _i32
    L.ds4a_paged_evict_shared.argtypes = L.ds4a_paged_evict.argtypes[:27] + [_vp] + L.ds4a_paged_evict.argtypes[27:]
    L.ds4a_paged_evict_shared.restype = _i32
    L.ds4a_add_rms_norm.argtypes = [_vp, _i32, _i64, _vp, _i32, _i64, _vp, _i64, _vp, _f32, _vp, _i32, _vp, _vp, _i32,
                                    _i32, _vp, _i32, _i32, _vp]
    L.ds4a_add_rms_norm.restype = _i32
    _lib = L
    return L


def _strerror(status):
    try:
        return load(build_if_missing=False).ds4a_strerror(status).decode()
    except Exception:
        return "?"


def _check(status, where):
    if status != DS4A_OK:
        raise Ds4aError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _req(t, name, dtype, dev=True):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if dev and not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


# ----------------------------------------------------------------------------
# Entry points (same names as the C ABI)
# ----------------------------------------------------------------------------

def ds4a_version():
    return load().ds4a_version()


def ds4a_workspace_bytes(op, U, Q, N_cap, top_k):
    n = load().ds4a_workspace_bytes(op, U, Q, N_cap, top_k)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("ds4a_workspace_bytes: sizes out of range")
    return n


def ds4a_get_device_status(stream=None):
    """(status, flags) after synchronising the stream; clears the device word."""
    flags = ctypes.c_uint(0)
    st = load().ds4a_get_device_status(_stream(stream), ctypes.byref(flags))
    return st, flags.value


def ds4a_debug_inject_error(code):
    load().ds4a_debug_inject_error(code)


def ds4a_debug_wait_timeout(limit_us, stream=None):
    """Device-side failure-path hook: a bounded wait that nothing completes
    gives up after limit_us and sets DS4A_DEV_TIMEOUT (no fault)."""
    _check(load().ds4a_debug_wait_timeout(int(limit_us), _stream(stream)), "ds4a_debug_wait_timeout")


def ds4a_indexer_score(iq, w, ik, n_rows, scores, q_pos=None, row_pos=None, stream=None):
    """iq bf16 [U,Q,64,128]; w f32 [U,Q,64]; ik bf16 [U,N_cap,128] (unit stride
    may exceed N_cap*128); n_rows i32 [U]; scores f32 [U,Q,N_cap] (written).
    q_pos i32 [U,Q] and row_pos i32 [U,N_cap] for a causal prefill chunk."""
    _req(iq, "iq", torch.bfloat16)
    _req(w, "w", torch.float32)
    _req(n_rows, "n_rows", torch.int32)
    _req(scores, "scores", torch.float32)
    if ik.dtype != torch.bfloat16 or not ik.is_cuda or ik.dim() != 3 or ik.stride(2) != 1 or ik.stride(1) != IDX_DIM:
        raise ValueError("ik: bf16 CUDA tensor [U, N_cap, 128] with contiguous rows")
    U, N_cap = ik.shape[0], ik.shape[1]
    Q = iq.shape[1]
    if iq.shape != (U, Q, N_IDX_HEAD, IDX_DIM) or w.shape != (U, Q, N_IDX_HEAD):
        raise ValueError("iq / w shape")
    if scores.shape != (U, Q, N_cap) or n_rows.shape != (U,):
        raise ValueError("scores / n_rows shape")
    if (q_pos is None) != (row_pos is None):
        raise ValueError("q_pos and row_pos go together")
    if q_pos is not None:
        _req(q_pos, "q_pos", torch.int32)
        _req(row_pos, "row_pos", torch.int32)
        if q_pos.shape != (U, Q) or row_pos.shape != (U, N_cap):
            raise ValueError("q_pos / row_pos shape")
    st = load().ds4a_indexer_score(_ptr(iq), _ptr(w), _ptr(ik), ik.stride(0), _ptr(n_rows), _ptr(q_pos),
                                   _ptr(row_pos), _ptr(scores), U, Q, N_cap, _stream(stream))
    _check(st, "ds4a_indexer_score")


def ds4a_topk_select(scores, n_rows, top_k, idx, count, ws, stream=None):
    """scores f32 [U,Q,N_cap]; n_rows i32 [U]; idx i32 [U,Q,top_k], count i32
    [U,Q] (written); ws uint8 CUDA tensor of ds4a_workspace_bytes(...) bytes."""
    _req(scores, "scores", torch.float32)
    _req(n_rows, "n_rows", torch.int32)
    _req(idx, "idx", torch.int32)
    _req(count, "count", torch.int32)
    U, Q, N_cap = scores.shape
    if idx.shape != (U, Q, top_k) or count.shape != (U, Q):
        raise ValueError("idx / count shape")
    st = load().ds4a_topk_select(_ptr(scores), _ptr(n_rows), U, Q, N_cap, top_k, _ptr(idx), _ptr(count), _ptr(ws),
                                 ws.numel() * ws.element_size() if ws is not None else 0, _stream(stream))
    _check(st, "ds4a_topk_select")


def ds4a_indexer_topk(iq, w, ik, n_rows, top_k, idx, count, ws, q_pos=None, row_pos=None, stream=None):
    """Indexer score and top-k select fused (no scores array): iq bf16
    [U,Q,64,128]; w f32 [U,Q,64]; ik bf16 [U,N_cap,128]; n_rows i32 [U]; idx
    i32 [U,Q,top_k] and count i32 [U,Q] (written); ws uint8 CUDA tensor of
    ds4a_workspace_bytes(DS4A_OP_INDEXER_TOPK, ...) bytes."""
    _req(iq, "iq", torch.bfloat16)
    _req(w, "w", torch.float32)
    _req(n_rows, "n_rows", torch.int32)
    _req(idx, "idx", torch.int32)
    _req(count, "count", torch.int32)
    if ik.dtype != torch.bfloat16 or not ik.is_cuda or ik.dim() != 3 or ik.stride(2) != 1 or ik.stride(1) != IDX_DIM:
        raise ValueError("ik: bf16 CUDA tensor [U, N_cap, 128] with contiguous rows")
    U, N_cap = ik.shape[0], ik.shape[1]
    Q = iq.shape[1]
    if iq.shape != (U, Q, N_IDX_HEAD, IDX_DIM) or w.shape != (U, Q, N_IDX_HEAD) or n_rows.shape != (U,):
        raise ValueError("iq / w / n_rows shape")
    if idx.shape != (U, Q, top_k) or count.shape != (U, Q):
        raise ValueError("idx / count shape")
    if (q_pos is None) != (row_pos is None):
        raise ValueError("q_pos and row_pos go together")
    if q_pos is not None:
        _req(q_pos, "q_pos", torch.int32)
        _req(row_pos, "row_pos", torch.int32)
        if q_pos.shape != (U, Q) or row_pos.shape != (U, N_cap):
            raise ValueError("q_pos / row_pos shape")
    st = load().ds4a_indexer_topk(_ptr(iq), _ptr(w), _ptr(ik), ik.stride(0), _ptr(n_rows), _ptr(q_pos), _ptr(row_pos),
                                  U, Q, N_cap, top_k, _ptr(idx), _ptr(count), _ptr(ws),
                                  ws.numel() * ws.element_size() if ws is not None else 0, _stream(stream))
    _check(st, "ds4a_indexer_topk")


def ds4a_topk_select_noalloc(scores, n_rows, top_k, idx, count, stream=None):
    """Same result as ds4a_topk_select, with no workspace argument: the scratch
    is the library's fixed 8 MiB device array.  For callers that cannot
    allocate device memory; calls on one device must not overlap on the GPU."""
    _req(scores, "scores", torch.float32)
    _req(n_rows, "n_rows", torch.int32)
    _req(idx, "idx", torch.int32)
    _req(count, "count", torch.int32)
    U, Q, N_cap = scores.shape
    if idx.shape != (U, Q, top_k) or count.shape != (U, Q):
        raise ValueError("idx / count shape")
    st = load().ds4a_topk_select_noalloc(_ptr(scores), _ptr(n_rows), U, Q, N_cap, top_k, _ptr(idx), _ptr(count),
                                         _stream(stream))
    _check(st, "ds4a_topk_select_noalloc")


def ds4a_sparse_attn_decode(q, rows, idx, count, raw, n_raw, scale, out, lse=None, ws=None, stream=None):
    """The 64-head call (see ds4a_sparse_attn_decode_heads)."""
    if q.dim() == 3 and q.shape[1] != N_HEAD:
        raise ValueError("q: 64 heads (use ds4a_sparse_attn_decode_heads for 128)")
    ds4a_sparse_attn_decode_heads(N_HEAD, q, rows, idx, count, raw, n_raw, scale, out, lse, ws, stream)


def ds4a_sparse_attn_decode_heads(n_head, q, rows, idx, count, raw, n_raw, scale, out, lse=None, ws=None,
                                  stream=None):
    """q bf16 [U,H,512] (H = 64, or 128 through ds4a_sparse_attn_decode_heads);
    rows bf16 [U,N_cap,512]; idx i32 [U,top_k]; count i32 [U]; raw fp16
    [U,128,512]; n_raw i32 [U]; out f32 [U,H,512]; lse f32 [U,H] or None; ws
    uint8 workspace or None."""
    _req(q, "q", torch.bfloat16)
    _req(idx, "idx", torch.int32)
    _req(count, "count", torch.int32)
    _req(n_raw, "n_raw", torch.int32)
    _req(out, "out", torch.float32)
    if rows.dtype != torch.bfloat16 or not rows.is_cuda or rows.dim() != 3 or rows.stride(2) != 1 \
            or rows.stride(1) != HEAD_DIM:
        raise ValueError("rows: bf16 CUDA tensor [U, N_cap, 512] with contiguous rows")
    if raw.dtype != torch.float16 or not raw.is_cuda or raw.dim() != 3 or raw.stride(2) != 1 \
            or raw.stride(1) != HEAD_DIM or raw.shape[1] != N_SWA:
        raise ValueError("raw: fp16 CUDA tensor [U, 128, 512] with contiguous rows")
    U = q.shape[0]
    top_k = idx.shape[1]
    if q.shape != (U, n_head, HEAD_DIM) or rows.shape[0] != U or idx.shape[0] != U or count.shape != (U,) \
            or raw.shape[0] != U or n_raw.shape != (U,) or out.shape != (U, n_head, HEAD_DIM):
        raise ValueError("shape mismatch")
    if lse is not None:
        _req(lse, "lse", torch.float32)
        if lse.shape != (U, n_head):
            raise ValueError("lse: [U, n_head]")
    st = load().ds4a_sparse_attn_decode_heads(int(n_head), _ptr(q), _ptr(rows), rows.stride(0), rows.shape[1], _ptr(idx),
                                        _ptr(count), top_k, _ptr(raw), raw.stride(0), _ptr(n_raw), float(scale),
                                        _ptr(out), _ptr(lse), U, _ptr(ws),
                                        ws.numel() * ws.element_size() if ws is not None else 0, _stream(stream))
    _check(st, "ds4a_sparse_attn_decode_heads")


def ds4a_dense_attn_decode(q, rows, n_rows, raw, n_raw, scale, out, lse=None, ws=None, stream=None):
    """The 64-head call (see ds4a_dense_attn_decode_heads)."""
    if q.dim() == 3 and q.shape[1] != N_HEAD:
        raise ValueError("q: 64 heads (use ds4a_dense_attn_decode_heads for 128)")
    ds4a_dense_attn_decode_heads(N_HEAD, q, rows, n_rows, raw, n_raw, scale, out, lse, ws, stream)


def ds4a_dense_attn_decode_heads(n_head, q, rows, n_rows, raw, n_raw, scale, out, lse=None, ws=None, stream=None):
    """q bf16 [U,64,512]; rows bf16 [U,N_cap,512]; n_rows i32 [U]; raw fp16
    [U,128,512]; n_raw i32 [U]; out f32 [U,64,512]; lse f32 [U,64] or None;
    ws uint8 workspace or None."""
    _req(q, "q", torch.bfloat16)
    _req(n_rows, "n_rows", torch.int32)
    _req(n_raw, "n_raw", torch.int32)
    _req(out, "out", torch.float32)
    if rows.dtype != torch.bfloat16 or not rows.is_cuda or rows.dim() != 3 or rows.stride(2) != 1 \
            or rows.stride(1) != HEAD_DIM:
        raise ValueError("rows: bf16 CUDA tensor [U, N_cap, 512] with contiguous rows")
    if raw.dtype != torch.float16 or not raw.is_cuda or raw.dim() != 3 or raw.stride(2) != 1 \
            or raw.stride(1) != HEAD_DIM or raw.shape[1] != N_SWA:
        raise ValueError("raw: fp16 CUDA tensor [U, 128, 512] with contiguous rows")
    U = q.shape[0]
    if q.shape != (U, n_head, HEAD_DIM) or rows.shape[0] != U or n_rows.shape != (U,) or raw.shape[0] != U \
            or n_raw.shape != (U,) or out.shape != (U, n_head, HEAD_DIM):
        raise ValueError("shape mismatch")
    if lse is not None:
        _req(lse, "lse", torch.float32)
        if lse.shape != (U, n_head):
            raise ValueError("lse: [U, n_head]")
    st = load().ds4a_dense_attn_decode_heads(int(n_head), _ptr(q), _ptr(rows), rows.stride(0), rows.shape[1], _ptr(n_rows), _ptr(raw),
                                       raw.stride(0), _ptr(n_raw), float(scale), _ptr(out), _ptr(lse), U, _ptr(ws),
                                       ws.numel() * ws.element_size() if ws is not None else 0, _stream(stream))
    _check(st, "ds4a_dense_attn_decode_heads")


def ds4a_sparse_attn_prefill(q, q_pos, rows, idx, count, raw, raw_pos0, scale, out, lse=None, ws=None, stream=None):
    """The 64-head call (see ds4a_sparse_attn_prefill_heads)."""
    if q.dim() == 3 and q.shape[1] != N_HEAD:
        raise ValueError("q: 64 heads (use ds4a_sparse_attn_prefill_heads for 128)")
    ds4a_sparse_attn_prefill_heads(N_HEAD, q, q_pos, rows, idx, count, raw, raw_pos0, scale, out, lse, ws, stream)


def ds4a_sparse_attn_prefill_heads(n_head, q, q_pos, rows, idx, count, raw, raw_pos0, scale, out, lse=None, ws=None,
                                   stream=None):
    """q bf16 [T,64,512]; q_pos i32 [T]; rows bf16 [N_cap,512]; idx i32
    [T,top_k]; count i32 [T]; raw fp16 [n_raw_rows,512] (row i = position
    raw_pos0 + i); out f32 [T,64,512]; lse f32 [T,64] or None."""
    _req(q, "q", torch.bfloat16)
    _req(q_pos, "q_pos", torch.int32)
    _req(rows, "rows", torch.bfloat16)
    _req(idx, "idx", torch.int32)
    _req(count, "count", torch.int32)
    _req(raw, "raw", torch.float16)
    _req(out, "out", torch.float32)
    T = q.shape[0]
    top_k = idx.shape[1]
    if q.shape != (T, n_head, HEAD_DIM) or q_pos.shape != (T,) or rows.dim() != 2 or rows.shape[1] != HEAD_DIM \
            or idx.shape[0] != T or count.shape != (T,) or raw.dim() != 2 or raw.shape[1] != HEAD_DIM \
            or out.shape != (T, n_head, HEAD_DIM):
        raise ValueError("shape mismatch")
    if lse is not None:
        _req(lse, "lse", torch.float32)
        if lse.shape != (T, n_head):
            raise ValueError("lse: [T, n_head]")
    st = load().ds4a_sparse_attn_prefill_heads(int(n_head), _ptr(q), _ptr(q_pos), _ptr(rows), rows.shape[0], _ptr(idx), _ptr(count),
                                         top_k, _ptr(raw), int(raw_pos0), raw.shape[0], float(scale), _ptr(out),
                                         _ptr(lse), T, _ptr(ws),
                                         ws.numel() * ws.element_size() if ws is not None else 0, _stream(stream))
    _check(st, "ds4a_sparse_attn_prefill_heads")


def ds4a_kv_push_raw(kv, raw, pos, n_raw, stream=None):
    """kv f32 [U,512]; raw fp16 [U,128,512] ring (written); pos i32 [U]; n_raw
    i32 [U] (written)."""
    _req(kv, "kv", torch.float32)
    _req(pos, "pos", torch.int32)
    _req(n_raw, "n_raw", torch.int32)
    if raw.dtype != torch.float16 or not raw.is_cuda or raw.dim() != 3 or raw.stride(2) != 1 \
            or raw.stride(1) != HEAD_DIM or raw.shape[1] != N_SWA:
        raise ValueError("raw: fp16 CUDA tensor [U, 128, 512] with contiguous rows")
    U = kv.shape[0]
    if kv.shape != (U, HEAD_DIM) or raw.shape[0] != U or pos.shape != (U,) or n_raw.shape != (U,):
        raise ValueError("shape mismatch")
    st = load().ds4a_kv_push_raw(_ptr(kv), _ptr(raw), raw.stride(0), _ptr(pos), _ptr(n_raw), U, _stream(stream))
    _check(st, "ds4a_kv_push_raw")


def ds4a_compressor_pool(kv, score, out, stream=None):
    """kv, score f32 [U,ratio,width]; out f32 [U,width] (written)."""
    _req(kv, "kv", torch.float32)
    _req(score, "score", torch.float32)
    _req(out, "out", torch.float32)
    if kv.dim() != 3 or score.shape != kv.shape or out.shape != (kv.shape[0], kv.shape[2]):
        raise ValueError("shape mismatch")
    U, ratio, width = kv.shape
    st = load().ds4a_compressor_pool(_ptr(kv), _ptr(score), ratio, width, _ptr(out), U, _stream(stream))
    _check(st, "ds4a_compressor_pool")


# ----------------------------------------------------------------------------
# FP8 row store
# ----------------------------------------------------------------------------

def _req_fp8_rows(rows8, row_scale, n_dims):
    if rows8.dtype != torch.uint8 or not rows8.is_cuda or rows8.dim() != n_dims or rows8.stride(-1) != 1 \
            or rows8.shape[-1] != HEAD_DIM or rows8.stride(-2) != HEAD_DIM:
        raise ValueError("rows8: uint8 CUDA tensor [..., N_cap, 512] of E4M3 codes with contiguous rows")
    if row_scale.dtype != torch.float32 or not row_scale.is_cuda or row_scale.stride(-1) != 1:
        raise ValueError("row_scale: float32 CUDA tensor, one scale per row")


def ds4a_rows_to_fp8(x, rows8, row_scale, stream=None):
    """x f32 [n,512] -> rows8 uint8 [n,512] E4M3 codes and row_scale f32 [n]
    (power-of-two scale per row), both written."""
    _req(x, "x", torch.float32)
    _req(rows8, "rows8", torch.uint8)
    _req(row_scale, "row_scale", torch.float32)
    n = x.shape[0]
    if x.shape != (n, HEAD_DIM) or rows8.shape != (n, HEAD_DIM) or row_scale.shape != (n,):
        raise ValueError("shape mismatch")
    st = load().ds4a_rows_to_fp8(_ptr(x), n, _ptr(rows8), _ptr(row_scale), _stream(stream))
    _check(st, "ds4a_rows_to_fp8")


def ds4a_sparse_attn_decode_fp8(q, rows8, row_scale, idx, count, raw, n_raw, scale, out, lse=None, ws=None,
                                stream=None):
    """ds4a_sparse_attn_decode with the compressed rows as the FP8 store:
    rows8 uint8 [U,N_cap,512] E4M3 codes, row_scale f32 [U,N_cap] laid out
    like the rows (unit u's scales start at u * rows8.stride(0) / 512)."""
    _req(q, "q", torch.bfloat16)
    _req(idx, "idx", torch.int32)
    _req(count, "count", torch.int32)
    _req(n_raw, "n_raw", torch.int32)
    _req(out, "out", torch.float32)
    _req_fp8_rows(rows8, row_scale, 3)
    if raw.dtype != torch.float16 or not raw.is_cuda or raw.dim() != 3 or raw.stride(2) != 1 \
            or raw.stride(1) != HEAD_DIM or raw.shape[1] != N_SWA:
        raise ValueError("raw: fp16 CUDA tensor [U, 128, 512] with contiguous rows")
    U, N_cap = rows8.shape[0], rows8.shape[1]
    top_k = idx.shape[1]
    if row_scale.dim() != 2 or row_scale.shape != (U, N_cap) or (U > 1 and
                                                               row_scale.stride(0) * HEAD_DIM != rows8.stride(0)):
        raise ValueError("row_scale: [U, N_cap] with unit stride rows8.stride(0) / 512")
    if q.shape != (U, N_HEAD, HEAD_DIM) or idx.shape[0] != U or count.shape != (U,) or raw.shape[0] != U \
            or n_raw.shape != (U,) or out.shape != (U, N_HEAD, HEAD_DIM):
        raise ValueError("shape mismatch")
    if lse is not None:
        _req(lse, "lse", torch.float32)
        if lse.shape != (U, N_HEAD):
            raise ValueError("lse: [U, 64]")
    st = load().ds4a_sparse_attn_decode_fp8(_ptr(q), _ptr(rows8), _ptr(row_scale), rows8.stride(0), N_cap, _ptr(idx),
                                            _ptr(count), top_k, _ptr(raw), raw.stride(0), _ptr(n_raw), float(scale),
                                            _ptr(out), _ptr(lse), U, _ptr(ws),
                                            ws.numel() * ws.element_size() if ws is not None else 0, _stream(stream))
    _check(st, "ds4a_sparse_attn_decode_fp8")


def ds4a_sparse_attn_prefill_fp8(q, q_pos, rows8, row_scale, idx, count, raw, raw_pos0, scale, out, lse=None,
                                 ws=None, stream=None):
    """ds4a_sparse_attn_prefill with the compressed rows as the FP8 store:
    rows8 uint8 [N_cap,512], row_scale f32 [N_cap]."""
    _req(q, "q", torch.bfloat16)
    _req(q_pos, "q_pos", torch.int32)
    _req(rows8, "rows8", torch.uint8)
    _req(row_scale, "row_scale", torch.float32)
    _req(idx, "idx", torch.int32)
    _req(count, "count", torch.int32)
    _req(raw, "raw", torch.float16)
    _req(out, "out", torch.float32)
    T = q.shape[0]
    top_k = idx.shape[1]
    if q.shape != (T, N_HEAD, HEAD_DIM) or q_pos.shape != (T,) or rows8.dim() != 2 or rows8.shape[1] != HEAD_DIM \
            or row_scale.shape != (rows8.shape[0],) or idx.shape[0] != T or count.shape != (T,) or raw.dim() != 2 \
            or raw.shape[1] != HEAD_DIM or out.shape != (T, N_HEAD, HEAD_DIM):
        raise ValueError("shape mismatch")
    if lse is not None:
        _req(lse, "lse", torch.float32)
        if lse.shape != (T, N_HEAD):
            raise ValueError("lse: [T, 64]")
    st = load().ds4a_sparse_attn_prefill_fp8(_ptr(q), _ptr(q_pos), _ptr(rows8), _ptr(row_scale), rows8.shape[0],
                                             _ptr(idx), _ptr(count), top_k, _ptr(raw), int(raw_pos0), raw.shape[0],
                                             float(scale), _ptr(out), _ptr(lse), T, _ptr(ws),
                                             ws.numel() * ws.element_size() if ws is not None else 0,
                                             _stream(stream))
    _check(st, "ds4a_sparse_attn_prefill_fp8")


# ----------------------------------------------------------------------------
# Paged caches
# ----------------------------------------------------------------------------

_I32, _F32, _F64, _BF16, _F16, _U8 = torch.int32, torch.float32, torch.float64, torch.bfloat16, torch.float16, torch.uint8
_TYPES = {torch.bfloat16: DS4A_BF16, torch.float16: DS4A_F16, torch.float32: DS4A_F32, torch.uint8: DS4A_E4M3}


# These calls are a few microseconds of GPU work, so the checks go by the cheap
# properties: the device's index and the element count (a contiguous tensor of
# the right count is the right memory whatever its shape).

def _req_ints(dev, *tensors):
    """Each (name, tensor, n) is contiguous int32 on device index `dev` with n elements."""
    for name, t, n in tensors:
        if t.dtype is not _I32 or t.get_device() != dev or t.numel() != n or not t.is_contiguous():
            raise ValueError(f"{name}: must be contiguous int32 on cuda:{dev} with {n} elements")


def _ints_ok(dev, n, *tensors):
    """Whether each is what _req_ints wants; the caller names them to it where one is not."""
    for t in tensors:
        if t.dtype is not _I32 or t.numel() != n or t.get_device() != dev or not t.is_contiguous():
            return False
    return True


def _table_stride(table, U, dev):
    if table.dtype is not _I32 or table.get_device() != dev or table.dim() != 2:
        raise ValueError(f"table: int32 [{U}, max_pages] on cuda:{dev}")
    n, cols = table.shape
    rows, one = table.stride()
    if n != U or cols < 1 or (cols > 1 and one != 1):
        raise ValueError(f"table: int32 [{U}, max_pages], entries of a row contiguous")
    return rows if U > 1 else cols, cols


def _device_index(t, name):
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name}: must be a CUDA tensor")
    return dev


def _opt(t):
    return None if t is None else t.data_ptr()


def _launch(dev, stream, name, *args):
    """Calls entry point `name` with device index `dev` current, on `stream` or that device's current stream."""
    f = getattr(_lib or load(), name)
    # torch.cuda.current_stream() builds a Stream object: 2.8 us of a 4 us call
    raw = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        st = f(*args, raw)
    else:
        with torch.cuda.device(dev):
            st = f(*args, raw)
    if st != DS4A_OK:
        raise Ds4aError(st, name)


def ds4a_paged_plan(past, add, ratio, page_size, free_pages, free_head, table, n_rows, n_raw, cu_tok, cu_row, tok_pos,
                    raw_slot, row_pos, row_slot, free_head_out, ring=None, stream=None, form=0, gone=None):
    """Block tables and slot maps of one step from the request lengths, all int32:
    past, add [B]; free_pages [n_free], free_head [1]; table [B, max_pages]
    (updated); n_rows, n_raw [B], cu_tok, cu_row [B + 1], tok_pos, raw_slot
    [T_cap], row_pos, row_slot [R_cap] and free_head_out [1] (written; may be
    free_head); ring [B] or None.  form: DS4A_PLAN_TOKENS_BY_SEQ and / or
    DS4A_PLAN_ROWS_BY_SEQ lay the token / row maps out by sequence (add 0 or 1),
    DS4A_PLAN_FIRST_POS makes row_pos the position of a row's first token.  gone [B]
    or None: each sequence's evicted rows (ds4a_paged_evict)."""
    dev = _device_index(past, "past")
    B, T, R, n_free = past.numel(), tok_pos.numel(), row_pos.numel(), free_pages.numel()
    _req_ints(dev, ("past", past, B), ("add", add, B), ("free_pages", free_pages, n_free), ("free_head", free_head, 1),
              ("free_head_out", free_head_out, 1), ("n_rows", n_rows, B), ("n_raw", n_raw, B), ("cu_tok", cu_tok, B + 1),
              ("cu_row", cu_row, B + 1), ("tok_pos", tok_pos, T), ("raw_slot", raw_slot, T), ("row_pos", row_pos, R),
              ("row_slot", row_slot, R))
    if ring is not None:
        _req_ints(dev, ("ring", ring, B))
    stride, max_pages = _table_stride(table, B, dev)
    name, lead, evicted = ("ds4a_paged_plan_form", (form,), ()) if form else ("ds4a_paged_plan", (), ())
    if gone is not None:
        _req_ints(dev, ("gone", gone, B))
        name, lead, evicted = "ds4a_paged_plan_evicted", (form,), (gone.data_ptr(),)
    _launch(dev, stream, name, *lead, past.data_ptr(), add.data_ptr(), *evicted, B, ratio, page_size, free_pages.data_ptr(), n_free,
            free_head.data_ptr(), free_head_out.data_ptr(), table.data_ptr(), stride, max_pages,
            _opt(ring), n_rows.data_ptr(), n_raw.data_ptr(), cu_tok.data_ptr(),
            cu_row.data_ptr(), tok_pos.data_ptr(), raw_slot.data_ptr(), T, row_pos.data_ptr(), row_slot.data_ptr(), R)


def ds4a_qk_norm_rope(q, k, pos, inv_freq, eps, q_weight, k_weight, q_out, k_out, k_slot=None, k_scale=None,
                      style=DS4A_ROPE_NEIGHBOURS, stream=None):
    """RMS norm and tail rotation of q [T,H,D] and of the key rows k [T,D] (bf16,
    fp16 or fp32; heads contiguous, any token stride; either may be None), D =
    512 or 128.  pos i32 [T] (negative: padding, nothing written); inv_freq f64
    [n_rot / 2]; q_weight, k_weight f32 [D] or None; q_out bf16 [T,H,D]
    (written); k_out [rows,D] bf16, fp16 or uint8 E4M3 codes with k_scale f32
    [rows] (row k_slot[t] written; k_slot i32 [T], None: row t)."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("q and k: at least one is needed")
    dev = _device_index(x, "q" if q is not None else "k")
    T, D = pos.numel(), x.shape[-1]
    H = q_type = k_type = k_out_type = q_stride = k_stride = k_rows = 0
    _req_ints(dev, ("pos", pos, T))
    if inv_freq.dtype is not _F64 or inv_freq.get_device() != dev or not inv_freq.is_contiguous():
        raise ValueError("inv_freq: contiguous float64 [n_rot / 2]")
    for w in (q_weight, k_weight):
        if w is not None and (w.dtype is not _F32 or w.get_device() != dev or w.numel() != D
                              or not w.is_contiguous()):
            raise ValueError(f"q_weight, k_weight: contiguous float32 [{D}]")
    if q is not None:
        q_type = _TYPES.get(q.dtype, -1)
        if not DS4A_BF16 <= q_type <= DS4A_F32 or q.dim() != 3:
            raise ValueError("q: bf16, fp16 or fp32 [T, H, D]")
        n, H, _ = q.shape
        q_stride, head, one = q.stride()
        if n != T or one != 1 or (H > 1 and head != D):
            raise ValueError("q: [T, H, D] with contiguous heads")
        if T <= 1:
            q_stride = H * D
        if q_out is None or q_out.dtype is not _BF16 or q_out.get_device() != dev \
                or q_out.numel() != T * H * D or not q_out.is_contiguous():
            raise ValueError("q_out: contiguous bf16 [T, H, D]")
    if k is not None:
        k_type = _TYPES.get(k.dtype, -1)
        if not DS4A_BF16 <= k_type <= DS4A_F32 or k.get_device() != dev or k.dim() != 2 or k.shape != (T, D):
            raise ValueError("k: bf16, fp16 or fp32 [T, D]")
        k_stride, one = k.stride()
        if one != 1:
            raise ValueError("k: contiguous rows")
        if T <= 1:
            k_stride = D
        k_out_type = _TYPES.get(None if k_out is None else k_out.dtype, -1)
        if k_out_type not in (DS4A_BF16, DS4A_F16, DS4A_E4M3) or k_out.get_device() != dev or k_out.dim() != 2 \
                or k_out.shape[1] != D or not k_out.is_contiguous():
            raise ValueError("k_out: contiguous bf16, fp16 or uint8 [rows, D]")
        k_rows = k_out.shape[0]
        if k_out_type == DS4A_E4M3 and (k_scale is None or k_scale.dtype is not _F32
                                        or k_scale.get_device() != dev or k_scale.numel() != k_rows
                                        or not k_scale.is_contiguous()):
            raise ValueError("k_scale: contiguous float32 [rows]")
        if k_slot is not None:
            _req_ints(dev, ("k_slot", k_slot, T))
    _launch(dev, stream, "ds4a_qk_norm_rope", _opt(q), q_type, q_stride, _opt(k), k_type, k_stride, pos.data_ptr(),
            inv_freq.data_ptr(), 2 * inv_freq.numel(), style, eps, _opt(q_weight), _opt(k_weight),
            q_out.data_ptr() if q is not None else None, k_out.data_ptr() if k is not None else None, k_out_type,
            k_scale.data_ptr() if k_out_type == DS4A_E4M3 else None, _opt(k_slot), k_rows, T, H, D)


def ds4a_paged_indexer_score(iq, w, ik, table, n_rows, scores, stream=None):
    """Indexer scores of one query per unit over paged keys: iq bf16 [U,1,64,128];
    w f32 [U,1,64]; ik bf16 [n_pages,P,128]; table i32 [U,max_pages]; n_rows i32
    [U]; scores f32 [U,1,N_cap] (written for r < n_rows[u])."""
    dev = _device_index(iq, "iq")
    if scores.dim() != 3:
        raise ValueError("scores: [U, 1, N_cap]")
    U, one, N_cap = scores.shape
    if one != 1 or scores.dtype is not _F32 or scores.get_device() != dev or not scores.is_contiguous():
        raise ValueError("scores: contiguous float32 [U, 1, N_cap]")
    if iq.dtype is not _BF16 or iq.numel() != U * N_IDX_HEAD * IDX_DIM or not iq.is_contiguous():
        raise ValueError("iq: contiguous bf16 [U, 1, 64, 128]")
    if w.dtype is not _F32 or w.get_device() != dev or w.numel() != U * N_IDX_HEAD or not w.is_contiguous():
        raise ValueError("w: contiguous float32 [U, 1, 64]")
    if ik.dtype is not _BF16 or ik.get_device() != dev or ik.dim() != 3 or not ik.is_contiguous():
        raise ValueError("ik: contiguous bf16 [n_pages, page_size, 128]")
    n_pages, page_size, width = ik.shape
    if width != IDX_DIM:
        raise ValueError("ik: contiguous bf16 [n_pages, page_size, 128]")
    _req_ints(dev, ("n_rows", n_rows, U))
    stride, max_pages = _table_stride(table, U, dev)
    _launch(dev, stream, "ds4a_paged_indexer_score", iq.data_ptr(), w.data_ptr(), ik.data_ptr(), n_pages, page_size,
            table.data_ptr(), stride, max_pages, n_rows.data_ptr(), scores.data_ptr(), U, N_cap)


def _paged_rows(q, rows, row_scale, table, n_rows, idx, count):
    """What the attention calls over paged rows share: (device, U, H, the arguments
    from n_head to n_rows, those of the list)."""
    dev, shape = _device_index(q, "q"), q.shape
    if q.dtype is not _BF16 or len(shape) != 3 or shape[2] != HEAD_DIM or not q.is_contiguous():
        raise ValueError("q: contiguous bf16 [U, H, 512]")
    U, H, _ = shape
    kind, shape, scale_ptr = rows.dtype, rows.shape, None
    fp8 = kind is _U8
    if not (fp8 or kind is _BF16) or rows.get_device() != dev or len(shape) != 3 or shape[2] != HEAD_DIM \
            or not rows.is_contiguous():
        raise ValueError("rows: contiguous bf16 or uint8 [n_pages, page_size, 512]")
    n_pages, page_size, _ = shape
    if fp8:
        if row_scale is None or row_scale.dtype is not _F32 or row_scale.get_device() != dev \
                or row_scale.numel() != n_pages * page_size or not row_scale.is_contiguous():
            raise ValueError("row_scale: contiguous float32 [n_pages, page_size]")
        scale_ptr = row_scale.data_ptr()
    stride, max_pages = _table_stride(table, U, dev)
    if idx is None:
        if count is not None:
            raise ValueError("idx and count go together")
        if not _ints_ok(dev, U, n_rows):
            _req_ints(dev, ("n_rows", n_rows, U))
        lists = None, None, 0
    else:
        if count is None:
            raise ValueError("idx and count go together")
        top_k = idx.shape[-1]
        if not (_ints_ok(dev, U, n_rows, count) and _ints_ok(dev, U * top_k, idx)):
            _req_ints(dev, ("n_rows", n_rows, U), ("idx", idx, U * top_k), ("count", count, U))
        lists = idx.data_ptr(), count.data_ptr(), top_k
    return dev, U, H, (H, q.data_ptr(), rows.data_ptr(), DS4A_E4M3 if fp8 else DS4A_BF16, scale_ptr, n_pages, page_size,
                       table.data_ptr(), stride, max_pages, n_rows.data_ptr()), lists


def _workspace(ws, dev):
    if ws is None:
        return None, 0
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("ws: a contiguous tensor on the same device")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _paged_attn(name, q, rows, table, n_rows, raw, n_raw, scale, out, lse, ws, idx, count, row_scale, ring, stream):
    dev, U, H, lead, lists = _paged_rows(q, rows, row_scale, table, n_rows, idx, count)
    if out.dtype is not _BF16 or out.get_device() != dev or out.numel() != U * H * HEAD_DIM \
            or not out.is_contiguous():
        raise ValueError("out: contiguous bf16 [U, H, 512]")
    shape = raw.shape
    if raw.dtype is not _F16 or raw.get_device() != dev or len(shape) != 3 or shape[1] != N_SWA or shape[2] != HEAD_DIM \
            or not raw.is_contiguous():
        raise ValueError("raw: contiguous fp16 [n_ring, 128, 512]")
    n_ring, ring_ptr, lse_ptr = shape[0], None, None
    if ring is not None:
        if not _ints_ok(dev, U, n_raw, ring):
            _req_ints(dev, ("n_raw", n_raw, U), ("ring", ring, U))
        ring_ptr = ring.data_ptr()
    else:
        if not _ints_ok(dev, U, n_raw):
            _req_ints(dev, ("n_raw", n_raw, U))
        if n_ring < U:
            raise ValueError("raw: a ring per unit, or give ring")
    if lse is not None:
        if lse.dtype is not _F32 or lse.get_device() != dev or lse.numel() != U * H or not lse.is_contiguous():
            raise ValueError("lse: contiguous float32 [U, H]")
        lse_ptr = lse.data_ptr()
    _launch(dev, stream, name, *lead, *lists, raw.data_ptr(), n_ring, ring_ptr, n_raw.data_ptr(), scale, out.data_ptr(),
            lse_ptr, U, *_workspace(ws, dev))


def ds4a_paged_attn_decode(q, rows, table, n_rows, raw, n_raw, scale, out, lse=None, ws=None, idx=None, count=None,
                           row_scale=None, ring=None, stream=None):
    """Attention of one new token per unit over paged rows and the raw window: q
    bf16 [U,H,512] (H = 64 or 128); rows bf16 [n_pages,P,512], or uint8 E4M3
    codes with row_scale f32 [n_pages,P]; table i32 [U,max_pages]; n_rows i32
    [U]; raw fp16 [n_ring,128,512]; n_raw i32 [U]; ring i32 [U] or None (ring u);
    idx i32 [U,top_k] and count i32 [U]: the listed rows only, None: all rows;
    out bf16 [U,H,512]; lse f32 [U,H] or None; ws uint8 workspace of
    ds4a_workspace_bytes(DS4A_OP_PAGED_ATTN_DECODE, U, 1, max_pages * P, top_k)."""
    _paged_attn("ds4a_paged_attn_decode", q, rows, table, n_rows, raw, n_raw, scale, out, lse, ws, idx, count, row_scale,
                ring, stream)


def ds4a_paged_attn_blocks(q, rows, table, n_rows, block_idx, block_count, raw, n_raw, scale, out, lse=None, ws=None,
                           row_scale=None, ring=None, stream=None):
    """ds4a_paged_attn_decode over the rows of listed blocks (pages of the unit's
    table): block_idx i32 [U,top_k], block_count i32 [U]; ws uint8 workspace of
    ds4a_workspace_bytes(DS4A_OP_PAGED_ATTN_BLOCKS, U, 1, top_k * P, 0)."""
    if block_idx is None or block_count is None:
        raise ValueError("block_idx and block_count: a list of blocks per unit")
    _paged_attn("ds4a_paged_attn_blocks", q, rows, table, n_rows, raw, n_raw, scale, out, lse, ws, block_idx, block_count,
                row_scale, ring, stream)


def ds4a_paged_attn_mass(q, rows, table, n_rows, scale, lse, mass, idx=None, count=None, blocks=False, row_scale=None,
                         tok_pos=None, stream=None):
    """Adds the weights that an attention gave each row, exp(scale q.x - lse) summed
    over the plane's 64 heads, to mass f32 [H/64,U,>= max_pages * P] (updated).
    lse f32 [U,H] from that attention; the other arguments are its own, idx and
    count naming blocks with blocks=True.  tok_pos i32 [U] or None: units whose entry
    is negative are left as they were."""
    dev, U, H, lead, lists = _paged_rows(q, rows, row_scale, table, n_rows, idx, count)
    if lse.dtype is not _F32 or lse.get_device() != dev or lse.numel() != U * H or not lse.is_contiguous():
        raise ValueError("lse: contiguous float32 [U, H]")
    if mass.dtype is not _F32 or mass.get_device() != dev or mass.dim() != 3 or not mass.is_contiguous() \
            or mass.shape[0] * N_HEAD != H or mass.shape[1] != U:
        raise ValueError("mass: contiguous float32 [H / 64, U, rows]")
    if tok_pos is not None:
        _req_ints(dev, ("tok_pos", tok_pos, U))
    _launch(dev, stream, "ds4a_paged_attn_mass", *lead, DS4A_LIST_BLOCKS if blocks else DS4A_LIST_ROWS, *lists, scale,
            lse.data_ptr(), _opt(tok_pos), mass.data_ptr(), mass.shape[2], U)


def _block_keys(block_keys, n_pages, dev):
    """Checks the keys of n_pages (None: as many as there are) pages; their number."""
    shape = block_keys.shape
    if len(shape) != 2 or shape[1] != IDX_DIM or block_keys.dtype is not _BF16 or block_keys.get_device() != dev \
            or not block_keys.is_contiguous() or (n_pages is not None and shape[0] != n_pages):
        raise ValueError("block_keys: contiguous bf16 [n_pages, 128]")
    return shape[0]


def ds4a_paged_block_keys(ik, table, n_rows, block_keys, n_blocks, first_row=None, cu_row=None, stream=None):
    """Mean indexer key of each block (page) that got rows: ik bf16 [n_pages,P,128];
    table i32 [B,max_pages]; n_rows i32 [B]; block_keys bf16 [n_pages,128]
    (updated); n_blocks i32 [B] (written).  The rows from first_row i32 [B] on, or
    the last cu_row[b+1] - cu_row[b] (cu_row i32 [B+1], the plan's), or all."""
    dev = _device_index(ik, "ik")
    if ik.dtype is not _BF16 or ik.dim() != 3 or ik.shape[2] != IDX_DIM or not ik.is_contiguous():
        raise ValueError("ik: contiguous bf16 [n_pages, page_size, 128]")
    n_pages, page_size, _ = ik.shape
    _block_keys(block_keys, n_pages, dev)
    B = n_rows.numel()
    stride, max_pages = _table_stride(table, B, dev)
    if not _ints_ok(dev, B, n_rows, n_blocks):
        _req_ints(dev, ("n_rows", n_rows, B), ("n_blocks", n_blocks, B))
    first = cu = None
    if first_row is not None:
        _req_ints(dev, ("first_row", first_row, B))
        first = first_row.data_ptr()
    if cu_row is not None:
        _req_ints(dev, ("cu_row", cu_row, B + 1))
        cu = cu_row.data_ptr()
    _launch(dev, stream, "ds4a_paged_block_keys", ik.data_ptr(), n_pages, page_size, table.data_ptr(), stride, max_pages,
            n_rows.data_ptr(), first, cu, block_keys.data_ptr(), n_blocks.data_ptr(), B)


def ds4a_paged_block_score(iq, w, block_keys, table, n_blocks, scores, n_first=0, n_last=0, stream=None):
    """Indexer scores of one query per unit over its blocks' mean keys: iq bf16
    [U,1,64,128]; w f32 [U,1,64]; block_keys bf16 [n_pages,128]; table i32
    [U,max_pages]; n_blocks i32 [U]; scores f32 [U,1,NB_cap] (written for b <
    n_blocks[u]; +inf for the first n_first and last n_last blocks, which a list of at
    least n_first + n_last then holds)."""
    dev = _device_index(iq, "iq")
    if scores.dim() != 3:
        raise ValueError("scores: [U, 1, NB_cap]")
    U, one, NB_cap = scores.shape
    if one != 1 or scores.dtype is not _F32 or scores.get_device() != dev or not scores.is_contiguous():
        raise ValueError("scores: contiguous float32 [U, 1, NB_cap]")
    if iq.dtype is not _BF16 or iq.numel() != U * N_IDX_HEAD * IDX_DIM or not iq.is_contiguous():
        raise ValueError("iq: contiguous bf16 [U, 1, 64, 128]")
    if w.dtype is not _F32 or w.get_device() != dev or w.numel() != U * N_IDX_HEAD or not w.is_contiguous():
        raise ValueError("w: contiguous float32 [U, 1, 64]")
    n_pages = _block_keys(block_keys, None, dev)
    _req_ints(dev, ("n_blocks", n_blocks, U))
    stride, max_pages = _table_stride(table, U, dev)
    _launch(dev, stream, "ds4a_paged_block_score", iq.data_ptr(), w.data_ptr(), block_keys.data_ptr(), n_pages,
            table.data_ptr(), stride, max_pages, n_blocks.data_ptr(), n_first, n_last, scores.data_ptr(), U, NB_cap)


def ds4a_paged_evict(mass, n_rows, table, rows, free_pages, free_head, keep, limit, mass_out, n_rows_out, table_out,
                     free_pages_out, free_head_out, ws, first=0, recent=0, row_scale=None, ik=None, n_shared=None,
                     gone=None, gone_out=None, first_row=None, stream=None, n_shared_out=None):
    """Cuts every sequence of more than `limit` rows to `keep`: its first `first`, its
    last `recent` and those of the greatest mass, copied to pages of the free list;
    the old pages go back to it.  mass f32 [planes,B,>= max_pages * P]; n_rows i32
    [B]; table i32 [B,max_pages]; rows bf16 or uint8 [n_pages,P,512] with row_scale
    f32 [n_pages,P], ik bf16 [n_pages,P,128] or None (all updated); free_pages i32
    [n_free], free_head i32 [1]; each *_out may be its input; n_shared, gone,
    gone_out, first_row i32 [B] or None; n_shared_out i32 [B] or None (written, with
    n_shared: 0 for the sequences cut, whose pages are their own now; a sequence cut
    again with its old number loses pages); ws uint8 workspace of
    ds4a_workspace_bytes(DS4A_OP_PAGED_EVICT, B, 1, max_pages * P, keep)."""
    dev = _device_index(mass, "mass")
    B, n_free, shape = n_rows.numel(), free_pages.numel(), mass.shape
    if len(shape) != 3 or shape[1] != B or mass_out.shape != shape:
        raise ValueError("mass, mass_out: contiguous float32 [planes, B, rows]")
    for t in (mass, mass_out):
        if t.dtype is not _F32 or t.get_device() != dev or not t.is_contiguous():
            raise ValueError("mass, mass_out: contiguous float32 [planes, B, rows]")
    fp8, rows_shape = rows.dtype is _U8, rows.shape
    if not (fp8 or rows.dtype is _BF16) or rows.get_device() != dev or len(rows_shape) != 3 or rows_shape[2] != HEAD_DIM \
            or not rows.is_contiguous():
        raise ValueError("rows: contiguous bf16 or uint8 [n_pages, page_size, 512]")
    n_pages, page_size, _ = rows_shape
    scale_ptr = ik_ptr = None
    if fp8:
        if row_scale is None or row_scale.dtype is not _F32 or row_scale.get_device() != dev \
                or row_scale.numel() != n_pages * page_size or not row_scale.is_contiguous():
            raise ValueError("row_scale: contiguous float32 [n_pages, page_size]")
        scale_ptr = row_scale.data_ptr()
    if ik is not None:
        if ik.dtype is not _BF16 or ik.get_device() != dev or ik.numel() != n_pages * page_size * IDX_DIM \
                or not ik.is_contiguous():
            raise ValueError("ik: contiguous bf16 [n_pages, page_size, 128]")
        ik_ptr = ik.data_ptr()
    stride, max_pages = layout = _table_stride(table, B, dev)
    if table_out is not table and _table_stride(table_out, B, dev) != layout:
        raise ValueError("table_out: laid out as table")
    if not (_ints_ok(dev, B, n_rows, n_rows_out) and _ints_ok(dev, n_free, free_pages, free_pages_out)
            and _ints_ok(dev, 1, free_head, free_head_out)):
        _req_ints(dev, ("n_rows", n_rows, B), ("n_rows_out", n_rows_out, B), ("free_pages", free_pages, n_free),
                  ("free_pages_out", free_pages_out, n_free), ("free_head", free_head, 1), ("free_head_out", free_head_out, 1))
    opt = [None] * 4
    for k, t in enumerate((n_shared, gone, gone_out, first_row)):
        if t is not None:
            if not _ints_ok(dev, B, t):
                _req_ints(dev, (("n_shared", "gone", "gone_out", "first_row")[k], t, B))
            opt[k] = t.data_ptr()
    name = "ds4a_paged_evict"
    if n_shared_out is not None:
        _req_ints(dev, ("n_shared_out", n_shared_out, B))
        if n_shared is None:
            raise ValueError("n_shared_out: with n_shared")
        name = "ds4a_paged_evict_shared"
        opt.insert(1, n_shared_out.data_ptr())
    ws_ptr, ws_bytes = _workspace(ws, dev)
    _launch(dev, stream, name, mass.data_ptr(), shape[0], shape[2], mass_out.data_ptr(),
            n_rows.data_ptr(), n_rows_out.data_ptr(), table.data_ptr(), table_out.data_ptr(), stride, max_pages, page_size,
            n_pages, B, keep, limit, first, recent, rows.data_ptr(), DS4A_E4M3 if fp8 else DS4A_BF16, scale_ptr, ik_ptr,
            free_pages.data_ptr(), free_pages_out.data_ptr(), n_free, free_head.data_ptr(), free_head_out.data_ptr(), *opt,
            ws_ptr, ws_bytes)


# ----------------------------------------------------------------------------
# Between layers
# ----------------------------------------------------------------------------

def _norm_rows(t, name, dev, shape, n):
    """(address, type, row stride) of n elements as [T, D] rows in 16 or 32 bits.  A contiguous
    tensor of the right count is the right memory whatever its shape."""
    kind = _TYPES.get(t.dtype, -1)
    if not DS4A_BF16 <= kind <= DS4A_F32 or t.get_device() != dev or t.numel() != n:
        raise ValueError(f"{name}: bf16, fp16 or fp32 [T, D] on cuda:{dev}")
    if t.is_contiguous():
        return t.data_ptr(), kind, shape[1]
    if t.shape != shape or t.stride(1) != 1:
        raise ValueError(f"{name}: [T, D] with contiguous rows")
    return t.data_ptr(), kind, t.stride(0) if shape[0] > 1 else shape[1]


def ds4a_add_rms_norm(x, weight, eps, out=None, residual=None, res_out=None, codes=None, scales=None, group=128,
                      scale_style=DS4A_SCALE_POW2, n_live=None, stream=None):
    """h = x + residual; y = h * weight / sqrt(mean h^2 + eps): x [T,D], residual
    [T,D] or None and res_out [T,D] (h; may be residual) in bf16, fp16 or fp32, rows
    any stride apart; weight f32 [D] or None; out [T,D] in 16 or 32 bits (may be x) and / or
    codes uint8 [T,D] E4M3 with scales f32 [T,ceil(D / group)] (written), a scale
    for every 32, 64 or 128 elements or (group = 0) for a row; n_live i32 [1] or
    None: rows from there on are left as they were."""
    dev = _device_index(x, "x")
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x: [T, D]")
    T, D = shape
    n = T * D
    x_ptr, x_type, x_stride = _norm_rows(x, "x", dev, shape, n)
    res_ptr = ro_ptr = out_ptr = w_ptr = codes_ptr = scales_ptr = live_ptr = None
    res_type = res_stride = ro_stride = out_type = 0
    if residual is not None:
        res_ptr, res_type, res_stride = _norm_rows(residual, "residual", dev, shape, n)
    if res_out is not None:
        ro_ptr, ro_type, ro_stride = _norm_rows(res_out, "res_out", dev, shape, n)
        if residual is None or ro_type != res_type:
            raise ValueError("res_out: with a residual, in its type")
    if out is not None:
        out_ptr, out_type, out_stride = _norm_rows(out, "out", dev, shape, n)
        if out_stride != D:
            raise ValueError("out: contiguous [T, D]")
    if weight is not None:
        if weight.dtype is not _F32 or weight.get_device() != dev or weight.numel() != D or not weight.is_contiguous():
            raise ValueError(f"weight: contiguous float32 [{D}]")
        w_ptr = weight.data_ptr()
    if (codes is None) != (scales is None):
        raise ValueError("codes and scales go together")
    if codes is not None:
        if codes.dtype is not _U8 or codes.get_device() != dev or codes.numel() != n or not codes.is_contiguous():
            raise ValueError("codes: contiguous uint8 [T, D]")
        groups = -(-D // group) if group > 0 else 1
        if scales.dtype is not _F32 or scales.get_device() != dev or scales.numel() != T * groups \
                or not scales.is_contiguous():
            raise ValueError(f"scales: contiguous float32 [T, {groups}]")
        codes_ptr, scales_ptr = codes.data_ptr(), scales.data_ptr()
    if n_live is not None:
        _req_ints(dev, ("n_live", n_live, 1))
        live_ptr = n_live.data_ptr()
    _launch(dev, stream, "ds4a_add_rms_norm", x_ptr, x_type, x_stride, res_ptr, res_type, res_stride, ro_ptr, ro_stride,
            w_ptr, eps, out_ptr, out_type, codes_ptr, scales_ptr, group, scale_style, live_ptr, T, D)
