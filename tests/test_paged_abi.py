"""Host-side refusals of the paged-cache entry points: bad arguments come back as
error codes before a device is touched.  CPU only: nothing is launched."""
import pytest

from deepseek_v4_sparse_indexer_gb300 import _binding as B

FAKE = 0x10000   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    return B.load()


def call(f, args, **change):
    names = list(args)
    vals = dict(args, **change)
    assert set(vals) == set(names)
    return f(*[vals[n] for n in names], None)


PLAN = dict(past=FAKE, add=FAKE, B=2, ratio=4, page_size=64, free_pages=FAKE, n_free=8, free_head=FAKE,
            free_head_out=FAKE, table=FAKE, table_stride=16, max_pages=16, ring=None, n_rows=FAKE, n_raw=FAKE,
            cu_tok=FAKE, cu_row=FAKE, tok_pos=FAKE, raw_slot=FAKE, T_cap=8, row_pos=FAKE, row_slot=FAKE, R_cap=8)
ROPE = dict(q=FAKE, q_type=B.DS4A_BF16, q_tok_stride=64 * 512, k=2 * FAKE, k_type=B.DS4A_F32, k_tok_stride=512, pos=FAKE,
            inv_freq=FAKE, n_rot=64, style=0, eps=1e-6, q_weight=None, k_weight=None, q_out=3 * FAKE, k_out=4 * FAKE,
            k_out_type=B.DS4A_F16, k_scale=None, k_slot=FAKE, k_out_rows=128, T=4, n_head=64, head_dim=512)
SCORE = dict(iq=FAKE, w=FAKE, ik=FAKE, n_pages=9, page_size=64, table=FAKE, table_stride=4, max_pages=4, n_rows=FAKE,
             scores=FAKE, U=2, N_cap=256)
ATTN = dict(n_head=64, q=FAKE, rows=FAKE, rows_type=B.DS4A_BF16, row_scale=None, n_pages=9, page_size=64, table=FAKE,
            table_stride=4, max_pages=4, n_rows=FAKE, idx=None, count=None, top_k=0, raw=FAKE, n_ring=2, ring=None,
            n_raw=FAKE, scale=0.04, out=FAKE, lse=None, U=2, ws=FAKE, ws_bytes=1 << 30)


@pytest.mark.parametrize("change", [
    dict(past=None), dict(add=None), dict(table=None), dict(free_head=None), dict(free_head_out=None), dict(n_rows=None),
    dict(n_raw=None), dict(cu_tok=None), dict(cu_row=None), dict(tok_pos=None), dict(raw_slot=None), dict(row_pos=None),
    dict(row_slot=None), dict(free_pages=None), dict(n_free=-1), dict(B=0), dict(B=B.DS4A_MAX_PLAN_SEQS + 1),
    dict(ratio=0), dict(page_size=4), dict(page_size=48), dict(page_size=8192), dict(page_size=-64), dict(max_pages=0),
    dict(table_stride=15), dict(T_cap=0), dict(R_cap=0)])
def test_plan_rejects(lib, change):
    assert call(lib.ds4a_paged_plan, PLAN, **change) == B.DS4A_EINVAL


@pytest.mark.parametrize("change", [
    dict(q=None, k=None), dict(pos=None), dict(inv_freq=None), dict(inv_freq=FAKE + 4), dict(T=-1), dict(style=2),
    dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(q=FAKE + 8), dict(q_out=None),
    dict(q_out=FAKE + 2), dict(n_head=0), dict(q_tok_stride=64 * 512 - 8), dict(q_tok_stride=64 * 512 + 4),
    dict(k=FAKE + 4), dict(k_out=None), dict(k_out=2 * FAKE), dict(k_out=FAKE + 8), dict(k_tok_stride=508),
    dict(k_tok_stride=514), dict(k_out_rows=-1), dict(k_slot=None, k_out_rows=3), dict(q_weight=FAKE + 4),
    dict(k_weight=FAKE + 8), dict(k_out_type=B.DS4A_E4M3), dict(k_out_type=B.DS4A_E4M3, k_scale=FAKE + 2),
    dict(q_out=FAKE, q_tok_stride=64 * 512 + 8), dict(q_out=FAKE, q_type=B.DS4A_F16), dict(n_head=1 << 30)])
def test_rope_rejects(lib, change):
    assert call(lib.ds4a_qk_norm_rope, ROPE, **change) == B.DS4A_EINVAL


@pytest.mark.parametrize("change", [
    dict(head_dim=256), dict(head_dim=0), dict(n_rot=24), dict(n_rot=8), dict(n_rot=256), dict(q_type=B.DS4A_E4M3),
    dict(k_type=B.DS4A_E4M3), dict(k_type=9), dict(k_out_type=B.DS4A_F32),
    dict(head_dim=128, k_out_type=B.DS4A_E4M3, k_scale=FAKE)])
def test_rope_unsupported(lib, change):
    assert call(lib.ds4a_qk_norm_rope, ROPE, **change) == B.DS4A_EUNSUPPORTED


def test_rope_of_no_token_launches_nothing(lib):
    assert call(lib.ds4a_qk_norm_rope, ROPE, T=0) == B.DS4A_OK


@pytest.mark.parametrize("change", [
    dict(iq=None), dict(w=None), dict(ik=None), dict(table=None), dict(n_rows=None), dict(scores=None), dict(n_pages=0),
    dict(page_size=0), dict(page_size=96), dict(max_pages=0), dict(table_stride=3), dict(U=0), dict(U=(1 << 24) + 1),
    dict(N_cap=0), dict(iq=FAKE + 8), dict(ik=FAKE + 2), dict(w=FAKE + 2), dict(scores=FAKE + 1), dict(n_pages=1 << 25),
    dict(max_pages=1 << 25, table_stride=1 << 25), dict(U=1 << 20, N_cap=1 << 24, max_pages=1 << 18, table_stride=1 << 18)])
def test_indexer_rejects(lib, change):
    assert call(lib.ds4a_paged_indexer_score, SCORE, **change) == B.DS4A_EINVAL


@pytest.mark.parametrize("change", [
    dict(q=None), dict(rows=None), dict(table=None), dict(n_rows=None), dict(raw=None), dict(n_raw=None), dict(out=None),
    dict(U=0), dict(page_size=4), dict(page_size=100), dict(idx=FAKE), dict(count=FAKE), dict(top_k=4),
    dict(idx=FAKE, count=FAKE), dict(idx=FAKE, count=FAKE, top_k=B.DS4A_MAX_TOP_K + 1), dict(n_pages=0), dict(n_ring=0),
    dict(max_pages=0), dict(table_stride=3), dict(q=FAKE + 8), dict(rows=FAKE + 2), dict(raw=FAKE + 4),
    dict(out=FAKE + 2), dict(rows_type=B.DS4A_E4M3), dict(rows_type=B.DS4A_E4M3, row_scale=FAKE + 1),
    dict(scale=float("nan")), dict(n_pages=1 << 25), dict(max_pages=1 << 25, table_stride=1 << 25), dict(n_ring=1 << 24),
    dict(U=1 << 26)])
def test_attention_rejects(lib, change):
    assert call(lib.ds4a_paged_attn_decode, ATTN, **change) == B.DS4A_EINVAL


@pytest.mark.parametrize("change", [dict(n_head=32), dict(n_head=0), dict(rows_type=B.DS4A_F16),
                                    dict(rows_type=B.DS4A_F32)])
def test_attention_unsupported(lib, change):
    assert call(lib.ds4a_paged_attn_decode, ATTN, **change) == B.DS4A_EUNSUPPORTED


@pytest.mark.parametrize("heads,flag", [(64, 0), (128, B.DS4A_OP_FLAG_128_HEADS)])
def test_attention_workspace(lib, heads, flag):
    need = B.ds4a_workspace_bytes(B.DS4A_OP_PAGED_ATTN_DECODE | flag, 2, 1, 256, 0)
    slot = 2 * 64 * 514 * 4 + 16          # two partials and one share record per CTA
    assert need == 2 * 9 * (heads // 64) * slot        # 2 units x (6 + 3) tiles of 48 rows
    for change in (dict(ws_bytes=need - 1), dict(ws=None), dict(ws=FAKE + 16)):
        assert call(lib.ds4a_paged_attn_decode, ATTN, n_head=heads, **change) == B.DS4A_EWORKSPACE
    most = 160 * slot
    assert B.ds4a_workspace_bytes(B.DS4A_OP_PAGED_ATTN_DECODE | flag, 640, 1, 8192, 0) == most
    assert B.ds4a_workspace_bytes(B.DS4A_OP_PAGED_ATTN_DECODE | flag, 640, 1, 8192, 512) == most
    for bad in ((0, 1, 64, 0), (1, 1, 0, 0), (1, 1, 64, B.DS4A_MAX_TOP_K + 1), (1, 1, 64, -1), (1 << 26, 1, 1 << 20, 0)):
        with pytest.raises(ValueError):
            B.ds4a_workspace_bytes(B.DS4A_OP_PAGED_ATTN_DECODE | flag, *bad)


@pytest.mark.parametrize("name,args", [("ds4a_paged_plan", PLAN), ("ds4a_qk_norm_rope", ROPE),
                                       ("ds4a_paged_indexer_score", SCORE), ("ds4a_paged_attn_decode", ATTN)])
def test_injected_error(lib, name, args):
    lib.ds4a_debug_inject_error(B.DS4A_ECUDA)
    assert call(getattr(lib, name), args) == B.DS4A_ECUDA
