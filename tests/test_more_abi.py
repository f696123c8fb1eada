"""Host-side refusals of the block, eviction and residual-norm entry points: bad
arguments come back as error codes before a device is touched.  CPU only."""
import pytest

from deepseek_v4_sparse_indexer_gb300 import _binding as B

FAKE = 0x10000   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    return B.load()


def call(f, args, **change):
    vals = dict(args, **change)
    assert set(vals) == set(args)
    return f(*[vals[n] for n in args], None)


PLAN = dict(form=0, past=FAKE, add=FAKE, gone=FAKE, B=2, ratio=4, page_size=64, free_pages=FAKE, n_free=8, free_head=FAKE,
            free_head_out=FAKE, table=FAKE, table_stride=16, max_pages=16, ring=None, n_rows=FAKE, n_raw=FAKE,
            cu_tok=FAKE, cu_row=FAKE, tok_pos=FAKE, raw_slot=FAKE, T_cap=8, row_pos=FAKE, row_slot=FAKE, R_cap=8)
KEYS = dict(ik=FAKE, n_pages=9, page_size=64, table=FAKE, table_stride=4, max_pages=4, n_rows=FAKE, first_row=None, cu_row=FAKE,
            block_keys=FAKE, n_blocks=FAKE, B=2)
SCORE = dict(iq=FAKE, w=FAKE, block_keys=FAKE, n_pages=9, table=FAKE, table_stride=4, max_pages=4, n_blocks=FAKE, n_first=0,
             n_last=1, scores=FAKE, U=2, NB_cap=4)
ATTN = dict(n_head=64, q=FAKE, rows=FAKE, rows_type=B.DS4A_BF16, row_scale=None, n_pages=9, page_size=64, table=FAKE,
            table_stride=4, max_pages=4, n_rows=FAKE, idx=FAKE, count=FAKE, top_k=2, raw=FAKE, n_ring=2, ring=None,
            n_raw=FAKE, scale=0.04, out=FAKE, lse=None, U=2, ws=FAKE, ws_bytes=1 << 30)
MASS = dict(n_head=64, q=FAKE, rows=FAKE, rows_type=B.DS4A_BF16, row_scale=None, n_pages=9, page_size=64, table=FAKE,
            table_stride=4, max_pages=4, n_rows=FAKE, list_kind=0, idx=None, count=None, top_k=0, scale=0.04, lse=FAKE,
            tok_pos=None, mass=FAKE, mass_stride=256, U=2)
EVICT = dict(mass=FAKE, n_planes=1, mass_stride=256, mass_out=FAKE, n_rows=FAKE, n_rows_out=FAKE, table=FAKE, table_out=FAKE,
             table_stride=4, max_pages=4, page_size=64, n_pages=9, B=2, keep=100, limit=128, first=4, recent=16, rows=FAKE,
             rows_type=B.DS4A_BF16, row_scale=None, ik=None, free_pages=FAKE, free_pages_out=FAKE, n_free=9, free_head=FAKE,
             free_head_out=FAKE, n_shared=None, gone=None, gone_out=None, first_row=None, ws=FAKE, ws_bytes=1 << 20)
NORM = dict(x=FAKE, x_type=B.DS4A_BF16, x_stride=4096, res=FAKE, res_type=B.DS4A_F32, res_stride=4096, res_out=FAKE,
            res_out_stride=4096, weight=None, eps=1e-6, out=FAKE, out_type=B.DS4A_BF16, codes=FAKE, scales=FAKE, group=128,
            scale_style=0, n_live=None, T=4, D=4096)


@pytest.mark.parametrize("change", [dict(gone=None), dict(past=None), dict(form=8), dict(B=0), dict(page_size=48),
                                    dict(table_stride=15), dict(form=1, T_cap=1)])
def test_plan_evicted_rejects(lib, change):
    assert call(lib.ds4a_paged_plan_evicted, PLAN, **change) == B.DS4A_EINVAL


@pytest.mark.parametrize("change", [
    dict(ik=None), dict(table=None), dict(n_rows=None), dict(block_keys=None), dict(n_blocks=None), dict(first_row=FAKE),
    dict(page_size=4), dict(page_size=96), dict(B=0), dict(B=B.DS4A_MAX_PLAN_SEQS + 1), dict(n_pages=0), dict(max_pages=0),
    dict(table_stride=3), dict(ik=FAKE + 8), dict(block_keys=FAKE + 2), dict(n_pages=1 << 25),
    dict(max_pages=1 << 25, table_stride=1 << 25), dict(B=8192, max_pages=1 << 18, table_stride=1 << 18, page_size=8)])
def test_block_keys_rejects(lib, change):
    assert call(lib.ds4a_paged_block_keys, KEYS, **change) == B.DS4A_EINVAL


@pytest.mark.parametrize("change", [
    dict(iq=None), dict(w=None), dict(block_keys=None), dict(table=None), dict(n_blocks=None), dict(scores=None),
    dict(n_first=-1), dict(n_last=-1), dict(U=0), dict(U=(1 << 24) + 1), dict(NB_cap=0), dict(n_pages=0), dict(max_pages=0),
    dict(table_stride=3), dict(iq=FAKE + 8), dict(block_keys=FAKE + 8), dict(w=FAKE + 2), dict(scores=FAKE + 1),
    dict(U=1 << 24, max_pages=1 << 20, table_stride=1 << 20, NB_cap=1 << 20)])
def test_block_score_rejects(lib, change):
    assert call(lib.ds4a_paged_block_score, SCORE, **change) == B.DS4A_EINVAL


@pytest.mark.parametrize("change", [
    dict(idx=None), dict(count=None), dict(top_k=0), dict(idx=None, count=None, top_k=0), dict(top_k=-1),
    dict(top_k=B.DS4A_MAX_TOP_K + 1), dict(q=None), dict(raw=None), dict(out=None), dict(n_raw=None), dict(n_ring=0),
    dict(page_size=100), dict(q=FAKE + 8), dict(rows_type=B.DS4A_E4M3), dict(scale=float("nan")), dict(U=0),
    dict(table_stride=3), dict(U=1 << 24, top_k=2048, page_size=4096, max_pages=64, table_stride=64)])
def test_attention_over_blocks_rejects(lib, change):
    assert call(lib.ds4a_paged_attn_blocks, ATTN, **change) == B.DS4A_EINVAL


@pytest.mark.parametrize("change", [
    dict(lse=None), dict(mass=None), dict(mass_stride=255), dict(mass=FAKE + 2), dict(lse=FAKE + 1), dict(list_kind=2),
    dict(idx=FAKE), dict(count=FAKE), dict(top_k=3), dict(idx=FAKE, count=FAKE), dict(q=None), dict(rows=None),
    dict(table=None), dict(n_rows=None), dict(rows_type=B.DS4A_E4M3), dict(U=0), dict(page_size=4)])
def test_mass_rejects(lib, change):
    assert call(lib.ds4a_paged_attn_mass, MASS, **change) == B.DS4A_EINVAL


@pytest.mark.parametrize("name,args", [("ds4a_paged_attn_blocks", ATTN), ("ds4a_paged_attn_mass", MASS)])
@pytest.mark.parametrize("change", [dict(n_head=32), dict(rows_type=B.DS4A_F16)])
def test_attention_unsupported(lib, name, args, change):
    assert call(getattr(lib, name), args, **change) == B.DS4A_EUNSUPPORTED


@pytest.mark.parametrize("change", [
    dict(mass=None), dict(mass_out=None), dict(n_rows=None), dict(n_rows_out=None), dict(table=None), dict(table_out=None),
    dict(rows=None), dict(free_head=None), dict(free_head_out=None), dict(free_pages=None), dict(free_pages_out=None),
    dict(n_free=-1), dict(n_planes=0), dict(n_planes=17), dict(mass_stride=255), dict(B=0), dict(B=B.DS4A_MAX_PLAN_SEQS + 1),
    dict(page_size=4), dict(max_pages=0), dict(table_stride=3), dict(n_pages=0), dict(keep=0), dict(keep=257, limit=300),
    dict(limit=99), dict(first=-1), dict(recent=-1), dict(first=50, recent=51), dict(first=2 ** 31 - 1, recent=2 ** 31 - 1),
    dict(rows=FAKE + 8), dict(ik=FAKE + 8), dict(mass=FAKE + 2), dict(rows_type=B.DS4A_E4M3), dict(gone=FAKE),
    dict(B=8192, max_pages=1 << 18, table_stride=1 << 18, mass_stride=1 << 24)])
def test_evict_rejects(lib, change):
    assert call(lib.ds4a_paged_evict, EVICT, **change) == B.DS4A_EINVAL


def test_evict_workspace_and_types(lib):
    need = B.ds4a_workspace_bytes(B.DS4A_OP_PAGED_EVICT, 2, 1, 256, 100)
    assert need == 4 * (64 + 2 + 2 * 13 + 2 * 100)          # pages of 8 rows at least
    for change in (dict(ws=None), dict(ws=FAKE + 16), dict(ws_bytes=4 * (64 + 2 + 2 * 2 + 200) - 1)):
        assert call(lib.ds4a_paged_evict, EVICT, **change) == B.DS4A_EWORKSPACE
    assert call(lib.ds4a_paged_evict, EVICT, rows_type=B.DS4A_F16) == B.DS4A_EUNSUPPORTED
    for bad in ((0, 1, 256, 100), (2, 1, 256, 0), (2, 1, 256, 257), (B.DS4A_MAX_PLAN_SEQS + 1, 1, 256, 100)):
        with pytest.raises(ValueError):
            B.ds4a_workspace_bytes(B.DS4A_OP_PAGED_EVICT, *bad)


@pytest.mark.parametrize("flag", [0, B.DS4A_OP_FLAG_128_HEADS])
def test_attention_workspace(lib, flag):
    """A list of blocks takes what as many rows take."""
    rows = B.ds4a_workspace_bytes(B.DS4A_OP_PAGED_ATTN_DECODE | flag, 3, 1, 2 * 64, 0)
    need = B.ds4a_workspace_bytes(B.DS4A_OP_PAGED_ATTN_BLOCKS | flag, 3, 1, 2 * 64, 0)
    assert need == rows > 0
    heads = 128 if flag else 64
    for change in (dict(ws_bytes=need - 1), dict(ws=None), dict(ws=FAKE + 16)):
        assert call(lib.ds4a_paged_attn_blocks, ATTN, U=3, n_head=heads, **change) == B.DS4A_EWORKSPACE
    with pytest.raises(ValueError):
        B.ds4a_workspace_bytes(B.DS4A_OP_PAGED_ATTN_BLOCKS | flag, 3, 1, 128, 2)


@pytest.mark.parametrize("change", [
    dict(x=None), dict(out=None, codes=None), dict(res=None), dict(scales=None), dict(scale_style=2), dict(eps=0.0),
    dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(x=FAKE + 8), dict(res=FAKE + 8), dict(out=FAKE + 4),
    dict(codes=FAKE + 8), dict(scales=FAKE + 2), dict(weight=FAKE + 4), dict(n_live=FAKE + 2), dict(T=-1),
    dict(x_stride=4088), dict(x_stride=4100), dict(res_stride=4095), dict(res_out_stride=4098), dict(res_out_stride=4104)])
def test_norm_rejects(lib, change):
    assert call(lib.ds4a_add_rms_norm, NORM, **change) == B.DS4A_EINVAL


@pytest.mark.parametrize("change", [dict(D=0), dict(D=4), dict(D=1001), dict(D=B.DS4A_MAX_NORM_DIM + 8), dict(x_type=3),
                                    dict(res_type=3), dict(out_type=3), dict(group=16), dict(group=-1), dict(group=256)])
def test_norm_unsupported(lib, change):
    assert call(lib.ds4a_add_rms_norm, NORM, **change) == B.DS4A_EUNSUPPORTED


def test_norm_of_no_row_launches_nothing(lib):
    assert call(lib.ds4a_add_rms_norm, NORM, T=0) == B.DS4A_OK


@pytest.mark.parametrize("name,args", [
    ("ds4a_paged_plan_evicted", PLAN), ("ds4a_paged_block_keys", KEYS), ("ds4a_paged_block_score", SCORE),
    ("ds4a_paged_attn_blocks", ATTN), ("ds4a_paged_attn_mass", MASS), ("ds4a_paged_evict", EVICT), ("ds4a_add_rms_norm", NORM)])
def test_injected_error(lib, name, args):
    lib.ds4a_debug_inject_error(B.DS4A_ECUDA)
    assert call(getattr(lib, name), args) == B.DS4A_ECUDA


def test_step_options():
    from deepseek_v4_sparse_indexer_gb300 import PagedDecodeStep
    for bad in (dict(blocks=4), dict(blocks=4, top_k=16), dict(top_k=0, evict=(64, 96, 4, 8))):
        with pytest.raises(ValueError):
            PagedDecodeStep(2, 8, 16, device="cpu", **bad)
    step = PagedDecodeStep(2, 8, 16, top_k=0, blocks=4, mass=True, evict=(64, 96, 4, 8), device="cpu")
    assert step.scores.shape == (2, 1, 8) and step.idx.shape == (2, 1, 4)
