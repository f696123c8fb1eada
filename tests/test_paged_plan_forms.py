"""The layouts of ds4a_paged_plan_form: refusals (CPU, nothing is launched), and on the
GPU each layout against the walk over the sequences."""
import random

import pytest
import torch

from deepseek_v4_sparse_indexer_gb300 import _binding as B
from paged_util import WINDOW, pages_of, plan_reference
from test_paged_abi import PLAN, call
from test_paged_plan_gpu import KEYS, Plan, status

TOKENS, ROWS, FIRST = B.DS4A_PLAN_TOKENS_BY_SEQ, B.DS4A_PLAN_ROWS_BY_SEQ, B.DS4A_PLAN_FIRST_POS


@pytest.mark.parametrize("form,change", [
    (16, {}), (-1, {}), (8 | TOKENS, {}), (TOKENS, dict(T_cap=1)), (ROWS, dict(R_cap=1)), (TOKENS | ROWS, dict(R_cap=1)),
    (TOKENS, dict(past=None)), (ROWS, dict(page_size=48)), (TOKENS, dict(B=B.DS4A_MAX_PLAN_SEQS + 1)), (0, dict(T_cap=0))])
def test_form_rejects(form, change):
    assert call(B.load().ds4a_paged_plan_form, dict(form=form, **PLAN), **change) == B.DS4A_EINVAL


def test_injected_error():
    B.load().ds4a_debug_inject_error(B.DS4A_ECUDA)
    assert call(B.load().ds4a_paged_plan_form, dict(form=TOKENS, **PLAN)) == B.DS4A_ECUDA


def by_sequence(p, form):
    """The walk's arrays, the maps of `form` laid out by sequence."""
    want, table, head = plan_reference(p.past, p.add, p.ratio, p.P, p.free, p.head, p.table, p.ring, p.T_cap, p.R_cap)
    if form & FIRST:
        want["row_pos"] = [x if x < 0 else x - (p.ratio - 1) for x in want["row_pos"]]
    for bit, cu, keys, cap in ((TOKENS, "cu_tok", ("tok_pos", "raw_slot"), p.T_cap),
                               (ROWS, "cu_row", ("row_pos", "row_slot"), p.R_cap)):
        if form & bit:
            for k in keys:
                have = [want[k][want[cu][b]] if want[cu][b + 1] > want[cu][b] else -1 for b in range(len(p.past))]
                want[k] = have + [-1] * (cap - len(have))
    return want, table, head


def go(lib, p, form, head_out=None):
    o = p.out
    lib.ds4a_paged_plan(p.d_past, p.d_add, p.ratio, p.P, p.d_free, p.d_head, p.d_table[:, :p.max_pages],
                        *[o[k] for k in KEYS], p.d_head_out if head_out is None else head_out, ring=p.d_ring, form=form)


def check(p, form):
    want, table, head = by_sequence(p, form)
    for k in KEYS:
        assert p.out[k].tolist() == want[k], k
        assert (p.room[k][:4 + p.off] == -77).all() and (p.room[k][-4:] == -77).all(), k
    assert p.d_table[:, :p.max_pages].tolist() == table
    return head


@pytest.mark.gpu
@pytest.mark.parametrize("form", [TOKENS, ROWS, TOKENS | ROWS, TOKENS | ROWS | FIRST])
@pytest.mark.parametrize("B_,ratio,P,off", [(1, 4, 64, 0), (3, 1, 8, 1), (130, 4, 8, 0), (130, 2, 4096, 1), (1500, 128, 16, 0),
                                            (8192, 3, 64, 0)])
def test_decode_steps(cuda_lib, B_, ratio, P, off, form):
    rng = random.Random(B_ + form)
    past = [rng.choice((0, rng.randint(0, 4000))) for _ in range(B_)]
    add = [rng.randint(0, 1) for _ in range(B_)]
    p = Plan(past, add, ratio, P, T_cap=B_ + rng.randint(0, 5), R_cap=B_ + rng.randint(0, 5), seed=B_, off=off)
    go(cuda_lib, p, form)
    assert status(cuda_lib) == (0, 0)
    assert p.d_head_out.item() == check(p, form)


@pytest.mark.gpu
@pytest.mark.parametrize("B_", [7, 8192])         # one CTA, and a cluster whose shared memory is at its largest
def test_head_in_place(cuda_lib, B_):
    p = Plan([3] * B_, [1] * B_, 4, 8, extra=0 if B_ == 7 else 600)
    go(cuda_lib, p, TOKENS | ROWS, head_out=p.d_head)
    assert status(cuda_lib) == (0, 0)
    assert p.d_head.item() == check(p, TOKENS | ROWS)


@pytest.mark.gpu
def test_more_than_one_token(cuda_lib):
    """Flagged, and as if the sequence had none."""
    p = Plan([8, 9, 3, 7], [1, 0, 1, 1], 4, 8, T_cap=4, R_cap=4)
    p.d_add[1] = 2
    go(cuda_lib, p, TOKENS | ROWS)
    assert status(cuda_lib) == (cuda_lib.DS4A_EDEVICE, cuda_lib.DS4A_DEV_BOUNDS)
    check(p, TOKENS | ROWS)


@pytest.mark.gpu
def test_captured_and_replayed(cuda_lib):
    p = Plan([0] * 9, [1] * 9, 4, 8, T_cap=9, R_cap=9, max_pages=20)
    go(cuda_lib, p, TOKENS | ROWS)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(cuda_lib, p, TOKENS | ROWS)
    rng = random.Random(2)
    for _ in range(4):
        past = [rng.randint(0, 400) for _ in range(9)]
        q = Plan(past, [rng.randint(0, 1) for _ in range(9)], 4, 8, T_cap=9, R_cap=9, max_pages=20, seed=sum(past))
        n = min(len(q.free), p.d_free.numel())
        for k in ("d_past", "d_add", "d_table", "d_ring"):
            getattr(p, k).copy_(getattr(q, k))
        p.d_free[:n].copy_(q.d_free[:n])
        q.free = p.d_free.tolist()
        graph.replay()
        q.out, q.room, q.d_table, q.off = p.out, p.room, p.d_table, p.off
        assert p.d_head_out.item() == check(q, TOKENS | ROWS)


@pytest.mark.gpu
def test_a_ring_or_page_that_is_not_there(cuda_lib):
    p = Plan([31, 31, 3], [1, 1, 1], 4, 8, T_cap=3, R_cap=3, free=[50], head=0)      # three new rows, one of a new page
    p.d_ring[2] = -1
    p.d_table[0, 0] = -1
    go(cuda_lib, p, TOKENS | ROWS)
    assert status(cuda_lib) == (cuda_lib.DS4A_EDEVICE, cuda_lib.DS4A_DEV_BOUNDS)
    assert p.out["raw_slot"].tolist() == [p.ring[0] * WINDOW + 31, p.ring[1] * WINDOW + 31, -1]
    assert p.out["row_slot"].tolist() == [-1, p.table[1][0] * 8 + 7, 50 * 8]
    assert p.out["tok_pos"].tolist() == [31, 31, 3] and p.out["row_pos"].tolist() == [31, 31, 3]


@pytest.mark.gpu
@pytest.mark.parametrize("ratio,P", [(1, 8), (4, 64), (128, 8)])
def test_first_position_of_a_chunk(cuda_lib, ratio, P):
    rng = random.Random(ratio)
    past = [rng.randint(0, 3000) for _ in range(40)]
    p = Plan(past, [rng.choice((0, 1, 129, rng.randint(0, 2048))) for _ in past], ratio, P)
    go(cuda_lib, p, FIRST)
    assert status(cuda_lib) == (0, 0)
    assert p.d_head_out.item() == check(p, FIRST)


@pytest.mark.gpu
@pytest.mark.parametrize("add", [40, 4000])       # one CTA, and every SM
def test_negative_head_takes_no_page(cuda_lib, add):
    """A head that was never set: flagged, and no page that another sequence may hold is handed out."""
    p = Plan([8, 0, 12], [add] * 3, 4, 8)
    p.d_head.fill_(-2)
    go(cuda_lib, p, 0)
    assert status(cuda_lib) == (cuda_lib.DS4A_EDEVICE, cuda_lib.DS4A_DEV_BOUNDS)
    assert p.d_head_out.item() == -2
    want, _, _ = by_sequence(p, 0)
    for k in ("n_rows", "n_raw", "cu_tok", "cu_row", "tok_pos", "raw_slot", "row_pos"):
        assert p.out[k].tolist() == want[k], k
    held = [1, 0, 1]
    slots = [p.table[b][j // 8] * 8 + j % 8 if j // 8 < held[b] else -1
             for b in range(3) for j in range(p.past[b] // 4, (p.past[b] + add) // 4)]
    assert p.out["row_slot"].tolist() == slots + [-1] * (p.R_cap - len(slots))
    new = [pages_of((p.past[b] + add) // 4, 8) for b in range(3)]
    assert p.d_table[:, :p.max_pages].tolist() == [p.table[b][:held[b]] + [-1] * (new[b] - held[b]) + p.table[b][new[b]:]
                                                   for b in range(3)]
