"""One pass of the three-tier compressed-attention step through the C ABI.

DecodeStep: U units (sequence x layer caches), one query each.
PrefillStep: one chunk of T queries of one sequence over a causal row store.
DenseStep: the ratio-128 layers' attention over all compressed rows (no
indexer, so no score or select).
ProducerStep: the cache producer at a ratio boundary: the raw-window push of
the new token, the compressor pooling of the frontier and (fp8=True) the FP8
store of the pooled row.

PagedDecodeStep: one decode step of a layer whose rows and keys lie in pages of a
shared pool, from the sequences' lengths and the layer's projections to the
attention output.

DecodeStep and PrefillStep with fp8=True read the compressed rows from the FP8
row store (x["rows8"] E4M3 codes, x["row_scale"] per-row scales) instead of
the bf16 rows; with fused=True they score and select in one call
(ds4a_indexer_topk: no scores array, the same selection).

Both own their outputs and workspaces (allocated once, reused every call, so a
call can be captured in a CUDA graph) and run indexer score -> top-k select ->
sparse attention on one CUDA stream, each op a C-ABI call into libds4a.so.
"""
import math

import torch

from . import _binding as B

DEFAULT_SCALE = 1.0 / math.sqrt(B.HEAD_DIM)


def _ws(nbytes, device):
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device) if nbytes else None


class DecodeStep:
    def __init__(self, U, N_cap, top_k=512, device="cuda", n_head=B.N_HEAD, fp8=False, fused=False):
        if fp8 and n_head != B.N_HEAD:
            raise ValueError("the FP8 row store is read with 64 query heads")
        self.U, self.N_cap, self.top_k, self.n_head, self.fp8, self.fused = U, N_cap, top_k, n_head, fp8, fused
        dev = torch.device(device)
        flag = B.DS4A_OP_FLAG_128_HEADS if n_head == 128 else 0
        self.scores = None if fused else torch.empty(U, 1, N_cap, dtype=torch.float32, device=dev)
        self.ws_fused = _ws(B.ds4a_workspace_bytes(B.DS4A_OP_INDEXER_TOPK, U, 1, N_cap, top_k), dev) if fused else None
        self.idx = torch.empty(U, 1, top_k, dtype=torch.int32, device=dev)
        self.count = torch.empty(U, 1, dtype=torch.int32, device=dev)
        self.out = torch.empty(U, n_head, B.HEAD_DIM, dtype=torch.float32, device=dev)
        self.lse = torch.empty(U, n_head, dtype=torch.float32, device=dev)
        self.ws_topk = None if fused else _ws(B.ds4a_workspace_bytes(B.DS4A_OP_TOPK_SELECT, U, 1, N_cap, top_k), dev)
        self.ws_attn = _ws(B.ds4a_workspace_bytes(B.DS4A_OP_SPARSE_ATTN_DECODE | flag, U, 1, N_cap, top_k), dev)

    def score(self, x, stream=None):
        iq, w = x["iq"].view(self.U, 1, B.N_IDX_HEAD, B.IDX_DIM), x["w"].view(self.U, 1, B.N_IDX_HEAD)
        if self.fused:
            B.ds4a_indexer_topk(iq, w, x["ik"], x["n_rows"], self.top_k, self.idx, self.count, self.ws_fused,
                                stream=stream)
            return
        B.ds4a_indexer_score(iq, w, x["ik"], x["n_rows"], self.scores, stream=stream)

    def select(self, x, stream=None):
        if self.fused:
            return                                   # done by score()
        B.ds4a_topk_select(self.scores, x["n_rows"], self.top_k, self.idx, self.count, self.ws_topk, stream=stream)

    def attend(self, x, scale=DEFAULT_SCALE, stream=None):
        idx, count = self.idx.view(self.U, self.top_k), self.count.view(self.U)
        if self.fp8:
            B.ds4a_sparse_attn_decode_fp8(x["q"], x["rows8"], x["row_scale"], idx, count, x["raw"], x["n_raw"], scale,
                                          self.out, self.lse, self.ws_attn, stream=stream)
            return
        B.ds4a_sparse_attn_decode_heads(self.n_head, x["q"], x["rows"], idx, count, x["raw"], x["n_raw"], scale,
                                        self.out, self.lse, self.ws_attn, stream=stream)

    def __call__(self, x, scale=DEFAULT_SCALE, stream=None):
        self.score(x, stream)
        self.select(x, stream)
        self.attend(x, scale, stream)
        return self.out


class PrefillStep:
    def __init__(self, T, N_cap, top_k=512, device="cuda", n_head=B.N_HEAD, fp8=False, fused=False):
        if fp8 and n_head != B.N_HEAD:
            raise ValueError("the FP8 row store is read with 64 query heads")
        self.T, self.N_cap, self.top_k, self.n_head, self.fp8, self.fused = T, N_cap, top_k, n_head, fp8, fused
        dev = torch.device(device)
        flag = B.DS4A_OP_FLAG_128_HEADS if n_head == 128 else 0
        self.scores = None if fused else torch.empty(1, T, N_cap, dtype=torch.float32, device=dev)
        self.ws_fused = _ws(B.ds4a_workspace_bytes(B.DS4A_OP_INDEXER_TOPK, 1, T, N_cap, top_k), dev) if fused else None
        self.idx = torch.empty(1, T, top_k, dtype=torch.int32, device=dev)
        self.count = torch.empty(1, T, dtype=torch.int32, device=dev)
        self.out = torch.empty(T, n_head, B.HEAD_DIM, dtype=torch.float32, device=dev)
        self.lse = torch.empty(T, n_head, dtype=torch.float32, device=dev)
        self.ws_topk = None if fused else _ws(B.ds4a_workspace_bytes(B.DS4A_OP_TOPK_SELECT, 1, T, N_cap, top_k), dev)
        self.ws_attn = _ws(B.ds4a_workspace_bytes(B.DS4A_OP_SPARSE_ATTN_PREFILL | flag, 1, T, N_cap, top_k), dev)

    def score(self, x, stream=None):
        T, N = self.T, self.N_cap
        iq, w = x["iq"].view(1, T, B.N_IDX_HEAD, B.IDX_DIM), x["w"].view(1, T, B.N_IDX_HEAD)
        ik, qp, rp = x["ik"].view(1, N, B.IDX_DIM), x["q_pos"].view(1, T), x["row_pos"].view(1, N)
        if self.fused:
            B.ds4a_indexer_topk(iq, w, ik, x["n_rows"], self.top_k, self.idx, self.count, self.ws_fused,
                                q_pos=qp, row_pos=rp, stream=stream)
            return
        B.ds4a_indexer_score(iq, w, ik, x["n_rows"], self.scores, q_pos=qp, row_pos=rp, stream=stream)

    def select(self, x, stream=None):
        if self.fused:
            return                                   # done by score()
        B.ds4a_topk_select(self.scores, x["n_rows"], self.top_k, self.idx, self.count, self.ws_topk, stream=stream)

    def attend(self, x, scale=DEFAULT_SCALE, stream=None):
        idx, count = self.idx.view(self.T, self.top_k), self.count.view(self.T)
        if self.fp8:
            B.ds4a_sparse_attn_prefill_fp8(x["q"], x["q_pos"], x["rows8"], x["row_scale"], idx, count, x["raw"],
                                           x["raw_pos0"], scale, self.out, self.lse, self.ws_attn, stream=stream)
            return
        B.ds4a_sparse_attn_prefill_heads(self.n_head, x["q"], x["q_pos"], x["rows"], idx, count, x["raw"],
                                         x["raw_pos0"], scale, self.out, self.lse, self.ws_attn, stream=stream)

    def __call__(self, x, scale=DEFAULT_SCALE, stream=None):
        self.score(x, stream)
        self.select(x, stream)
        self.attend(x, scale, stream)
        return self.out


class DenseStep:
    def __init__(self, U, N_cap, device="cuda", n_head=B.N_HEAD):
        self.U, self.N_cap, self.n_head = U, N_cap, n_head
        dev = torch.device(device)
        flag = B.DS4A_OP_FLAG_128_HEADS if n_head == 128 else 0
        self.out = torch.empty(U, n_head, B.HEAD_DIM, dtype=torch.float32, device=dev)
        self.lse = torch.empty(U, n_head, dtype=torch.float32, device=dev)
        self.ws_attn = _ws(B.ds4a_workspace_bytes(B.DS4A_OP_DENSE_ATTN_DECODE | flag, U, 1, N_cap, 0), dev)

    def attend(self, x, scale=DEFAULT_SCALE, stream=None):
        B.ds4a_dense_attn_decode_heads(self.n_head, x["q"], x["rows"], x["n_rows"], x["raw"], x["n_raw"], scale,
                                       self.out, self.lse, self.ws_attn, stream=stream)

    def __call__(self, x, scale=DEFAULT_SCALE, stream=None):
        self.attend(x, scale, stream)
        return self.out


class ProducerStep:
    def __init__(self, U, width=B.HEAD_DIM, device="cuda", fp8=False):
        if fp8 and width != B.HEAD_DIM:
            raise ValueError("the FP8 row store holds 512-wide rows")
        self.U, self.width, self.fp8 = U, width, fp8
        dev = torch.device(device)
        self.out = torch.empty(U, width, dtype=torch.float32, device=dev)
        self.rows8 = torch.empty(U, width, dtype=torch.uint8, device=dev) if fp8 else None
        self.row_scale = torch.empty(U, dtype=torch.float32, device=dev) if fp8 else None

    def push(self, x, stream=None):
        B.ds4a_kv_push_raw(x["row"], x["raw"], x["pos"], x["n_raw"], stream=stream)

    def pool(self, x, stream=None):
        B.ds4a_compressor_pool(x["kv"], x["score"], self.out, stream=stream)

    def store_fp8(self, stream=None):
        B.ds4a_rows_to_fp8(self.out, self.rows8, self.row_scale, stream=stream)

    def __call__(self, x, stream=None):
        self.push(x, stream)
        self.pool(x, stream)
        if self.fp8:
            self.store_fp8(stream)
        return self.out


class PagedDecodeStep:
    """One new token for each of up to U sequences, over paged caches.

    x holds, per step: past, add (i32 [U]: tokens in the cache and new ones, 1 or
    0, in any order; what out holds for a sequence without a new token is of no
    use unless it is empty: zeros), q [U,H,512] and kv [U,512], the projections
    before norm and rotation (bf16, fp16 or fp32); with top_k also iq [U,64,128]
    (with rotate_iq=False the indexer's queries as they are scored, bf16 and
    contiguous: for a model that does not normalise them) and w f32 [U,64].  And,
    kept by the program: table i32 [U,max_pages], free_pages and free_head
    (updated in place), ring i32 [U] or None, raw fp16 [n_ring,128,512], rows bf16
    [n_pages,P,512] (fp8: uint8 codes and row_scale f32 [n_pages,P]), ik bf16
    [n_pages,P,128] with top_k, inv_freq f64 [n_rot / 2], the norm weights q_norm,
    kv_norm, iq_norm, ik_norm (f32 or None) and, where the pooled rows have a norm
    of their own, row_norm (else they take kv_norm).

    style and idx_style (style unless given) say which dims pair in the layer's
    heads and rows and in the indexer's queries and keys.  A layer of `ratio`
    tokens per row finishes a row every ratio tokens: pooled [U,512] (and
    pooled_ik [U,128]) hold the rows finished in this step, new row i of the batch
    in row i (cu_row says whose) or, with pooled_by_sequence, sequence u's in row
    u, as ds4a_compressor_pool writes them (a sequence that finishes none: its row
    is not read).  row_position: "last" or "first", the token of a row whose
    position its tail (and its key's) is turned by.

    plan -> rotate -> store -> score -> select -> attend, each one call of the
    library (two for the indexer's part); outputs and workspaces are kept, so the
    step can be captured in a CUDA graph and replayed on other lengths.  top_k = 0:
    every row is attended to (the ratio-128 layers).
    """

    def __init__(self, U, max_pages, page_size, top_k=512, ratio=4, device="cuda", n_head=B.N_HEAD, fp8=False, eps=1e-6,
                 style=B.DS4A_ROPE_NEIGHBOURS, pooled_by_sequence=False, row_position="last", idx_style=None,
                 rotate_iq=True):
        self.U, self.page_size, self.top_k, self.ratio, self.n_head = U, page_size, top_k, ratio, n_head
        self.fp8, self.eps, self.style = fp8, eps, style
        self.idx_style = style if idx_style is None else idx_style
        self.rotate_iq = rotate_iq
        # q, kv and out are kept by sequence, so the tokens' positions and slots are too
        if row_position not in ("last", "first"):
            raise ValueError("row_position: \"last\" or \"first\"")
        self.form = B.DS4A_PLAN_TOKENS_BY_SEQ | (B.DS4A_PLAN_ROWS_BY_SEQ if pooled_by_sequence else 0) \
            | (B.DS4A_PLAN_FIRST_POS if row_position == "first" else 0)
        dev = torch.device(device)
        N_cap = max_pages * page_size
        flag = B.DS4A_OP_FLAG_128_HEADS if n_head == 128 else 0
        self.n_rows, self.n_raw, self.tok_pos, self.raw_slot, self.row_pos, self.row_slot = (
            torch.empty(U, dtype=torch.int32, device=dev) for _ in range(6))
        self.cu_tok, self.cu_row = (torch.empty(U + 1, dtype=torch.int32, device=dev) for _ in range(2))
        # rows of q without a token are left as they were, so they start as zeros
        self.q = torch.zeros(U, n_head, B.HEAD_DIM, dtype=torch.bfloat16, device=dev)
        self.out = torch.empty(U, n_head, B.HEAD_DIM, dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty(U, n_head, dtype=torch.float32, device=dev)
        self.ws_attn = _ws(B.ds4a_workspace_bytes(B.DS4A_OP_PAGED_ATTN_DECODE | flag, U, 1, N_cap, top_k), dev)
        self.idx = self.count = None
        if top_k:
            if rotate_iq:
                self.iq = torch.zeros(U, B.N_IDX_HEAD, B.IDX_DIM, dtype=torch.bfloat16, device=dev)
            self.scores = torch.empty(U, 1, N_cap, dtype=torch.float32, device=dev)
            self.idx = torch.empty(U, 1, top_k, dtype=torch.int32, device=dev)
            self.count = torch.empty(U, 1, dtype=torch.int32, device=dev)
            self.ws_topk = _ws(B.ds4a_workspace_bytes(B.DS4A_OP_TOPK_SELECT, U, 1, N_cap, top_k), dev)

    def plan(self, x, stream=None):
        B.ds4a_paged_plan(x["past"], x["add"], self.ratio, self.page_size, x["free_pages"], x["free_head"], x["table"],
                          self.n_rows, self.n_raw, self.cu_tok, self.cu_row, self.tok_pos, self.raw_slot, self.row_pos,
                          self.row_slot, x["free_head"], ring=x.get("ring"), stream=stream, form=self.form)

    def rotate(self, x, stream=None):
        B.ds4a_qk_norm_rope(x["q"], x["kv"], self.tok_pos, x["inv_freq"], self.eps, x.get("q_norm"), x.get("kv_norm"), self.q,
                            x["raw"].view(-1, B.HEAD_DIM), k_slot=self.raw_slot, style=self.style, stream=stream)
        if self.top_k and self.rotate_iq:
            B.ds4a_qk_norm_rope(x["iq"], None, self.tok_pos, x["inv_freq"], self.eps, x.get("iq_norm"), None, self.iq, None,
                                style=self.idx_style, stream=stream)

    def store(self, x, stream=None):
        row_norm = x["row_norm"] if "row_norm" in x else x.get("kv_norm")
        B.ds4a_qk_norm_rope(None, x["pooled"], self.row_pos, x["inv_freq"], self.eps, None, row_norm, None,
                            x["rows"].view(-1, B.HEAD_DIM), k_slot=self.row_slot,
                            k_scale=x["row_scale"].view(-1) if self.fp8 else None, style=self.style, stream=stream)
        if self.top_k:
            B.ds4a_qk_norm_rope(None, x["pooled_ik"], self.row_pos, x["inv_freq"], self.eps, None, x.get("ik_norm"), None,
                                x["ik"].view(-1, B.IDX_DIM), k_slot=self.row_slot, style=self.idx_style, stream=stream)

    def score(self, x, stream=None):
        iq = self.iq if self.rotate_iq else x["iq"]
        B.ds4a_paged_indexer_score(iq.view(self.U, 1, B.N_IDX_HEAD, B.IDX_DIM), x["w"].view(self.U, 1, B.N_IDX_HEAD),
                                   x["ik"], x["table"], self.n_rows, self.scores, stream=stream)

    def select(self, x, stream=None):
        with torch.cuda.device(self.scores.device):        # the paged calls see to it themselves
            B.ds4a_topk_select(self.scores, self.n_rows, self.top_k, self.idx, self.count, self.ws_topk, stream=stream)

    def attend(self, x, scale=DEFAULT_SCALE, stream=None):
        idx, count = (self.idx.view(self.U, self.top_k), self.count.view(self.U)) if self.top_k else (None, None)
        B.ds4a_paged_attn_decode(self.q, x["rows"], x["table"], self.n_rows, x["raw"], self.n_raw, scale, self.out, self.lse,
                                 self.ws_attn, idx=idx, count=count, row_scale=x["row_scale"] if self.fp8 else None,
                                 ring=x.get("ring"), stream=stream)

    def __call__(self, x, scale=DEFAULT_SCALE, stream=None):
        self.plan(x, stream)
        self.rotate(x, stream)
        self.store(x, stream)
        if self.top_k:
            self.score(x, stream)
            self.select(x, stream)
        self.attend(x, scale, stream)
        return self.out
