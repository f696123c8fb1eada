"""Sequences that share pages and are cut more than once: after its first cut a sequence's
pages are its own, and all of them go back to the list at the next one."""
import pytest
import torch

from paged_util import DEV, WINDOW, gen, ints, pages_of
from test_evict_gpu import Cache, status

pytestmark = pytest.mark.gpu


def cut(lib, c, n_shared, n_shared_out, keep, limit):
    ws = torch.empty(lib.ds4a_workspace_bytes(lib.DS4A_OP_PAGED_EVICT, c.B, 1, c.max_pages * c.P, keep), dtype=torch.uint8,
                     device=DEV)
    lib.ds4a_paged_evict(c.mass, c.n_rows, c.table, c.rows, c.free_pages, c.free_head, keep, limit, c.mass, c.n_rows, c.table,
                         c.free_pages, c.free_head, ws, ik=c.ik, gone=c.gone, gone_out=c.gone, n_shared=n_shared,
                         n_shared_out=n_shared_out)


@pytest.mark.parametrize("in_place", [True, False])
def test_cut_twice(cuda_lib, in_place):
    c = Cache([500, 300, 40, 500], 16, n_free=200)
    c.table[3, :20] = c.table[0, :20]
    first = c.table.tolist()
    shared = ints([20, 0, 2, 20])
    out = shared if in_place else torch.full_like(shared, 77)
    cut(cuda_lib, c, shared, out, 200, 250)
    status(cuda_lib)
    assert out.tolist() == [0, 0, 2, 0] and shared.tolist() == ([0, 0, 2, 0] if in_place else [20, 0, 2, 20])
    second = c.table.tolist()
    assert c.n_rows.tolist() == [200, 200, 40, 200]
    again = torch.full_like(out, 77)
    cut(cuda_lib, c, out, again, 100, 150)
    status(cuda_lib)
    assert again.tolist() == [0, 0, 2, 0] and c.n_rows.tolist() == [100, 100, 40, 100]
    listed = c.free_pages.tolist()[c.free_head.item():]
    assert len(set(listed)) == len(listed)
    for b, n in enumerate([500, 300, 40, 500]):
        if b == 2:
            continue
        own = first[b][20 if b in (0, 3) else 0:pages_of(n, 16)]             # what the first cut gave back
        assert set(second[b][:pages_of(200, 16)]) <= set(listed)             # and the second: every page
        # (a page that came back may have been taken again since)
        now = set(c.table[b, :pages_of(100, 16)].tolist())
        taken = set().union(*(set(c.table[k, :pages_of(100, 16)].tolist()) for k in (0, 1, 3)))
        assert set(own) <= set(listed) | taken and not now & set(listed)
    assert not set(first[0][:20]) & set(listed)                              # shared pages: the program's


def test_shared_of_a_large_batch_in_place(cuda_lib):
    """Every block reads the old numbers, the last one writes: 8,192 sequences, again and again."""
    lengths = [40 if b % 3 == 0 else 20 for b in range(8192)]
    c = Cache(lengths, 8, 1, ik=False, max_pages=8)
    back = 0
    keep = {k: getattr(c, k).clone() for k in ("mass", "n_rows", "table", "free_pages", "free_head", "gone")}
    for _ in range(20):
        for k, v in keep.items():
            getattr(c, k).copy_(v)
        shared = ints([b % 4 for b in range(8192)])
        cut(cuda_lib, c, shared, shared, 16, 32)
        status(cuda_lib)
        assert shared.tolist() == [0 if b % 3 == 0 else b % 4 for b in range(8192)]
        back = sum(5 - b % 4 for b in range(0, 8192, 3))
        assert c.free_head.item() == int(keep["free_head"]) + 2 * len(range(0, 8192, 3)) - back
    # refused: nothing is cut, nothing changes
    for k, v in keep.items():
        getattr(c, k).copy_(v)
    c.free_head.fill_(-1)
    shared = ints([b % 4 for b in range(8192)])
    cut(cuda_lib, c, shared, shared, 16, 32)
    status(cuda_lib, True)
    assert shared.tolist() == [b % 4 for b in range(8192)]


def test_steps_of_sequences_that_share_pages(cuda_lib):
    """Captured steps and evictions of three sequences, two of which begin with the same pages."""
    import deepseek_v4_sparse_indexer_gb300 as pkg
    U, P, max_pages, n_pages, scale = 3, 8, 4, 30, 512 ** -0.5
    g = gen(5)
    past = [19, 22, 17]
    table = [[0, 1, 2, -1], [0, 1, 3, -1], [4, 5, 6, -1]]
    free = list(range(7)) + list(range(7, n_pages))
    x = dict(table=ints(table), free_pages=ints(free), free_head=ints([7]), past=ints(past), add=ints([1] * U), gone=ints([0] * U),
             n_shared=ints([2, 2, 0]), mass=torch.zeros(1, U, max_pages * P, device=DEV),
             raw=torch.randn(U, WINDOW, 512, generator=g, device=DEV).to(torch.float16),
             rows=torch.randn(n_pages, P, 512, generator=g, device=DEV).to(torch.bfloat16),
             inv_freq=10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64, device=DEV) / 64))
    for k, shape in (("q", (U, 64, 512)), ("kv", (U, 512)), ("pooled", (U, 512))):
        x[k] = torch.randn(*shape, generator=g, device=DEV)
    step = pkg.PagedDecodeStep(U, max_pages, P, top_k=0, ratio=1, pooled_by_sequence=True, mass=True, evict=(16, 24, 1, 4))
    lengths, shared, cuts, graphs = list(past), [2, 2, 0], [0] * U, None
    for n in range(40):
        x["past"].copy_(ints([p + n for p in past]))
        if n < 2:
            step(x, scale), step.evict(x)
            if n == 1:
                torch.cuda.synchronize()
                graphs = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graphs):
                    step(x, scale), step.evict(x)
        else:
            graphs.replay()
        status(cuda_lib)
        for u in range(U):
            lengths[u] += 1
            if lengths[u] > 24:
                lengths[u], shared[u], cuts[u] = 16, 0, cuts[u] + 1
        assert step.n_rows.tolist() == lengths and x["n_shared"].tolist() == shared
        # every page is in the list or in one table, once; the shared ones in none that was cut
        mine = [p for u in range(U) for p in x["table"][u, shared[u]:pages_of(lengths[u], P)].tolist()]
        listed = x["free_pages"].tolist()[x["free_head"].item():]
        assert sorted(mine + listed + [0, 1]) == list(range(n_pages))
        for u in range(U):
            assert x["table"][u, :shared[u]].tolist() == [0, 1][:shared[u]]
    assert min(cuts) >= 3


def test_rejects_other_tensors(cuda_lib):
    c = Cache([100, 64], 16)
    for bad in (ints([0]), torch.zeros(2, device=DEV), torch.zeros(2, dtype=torch.int32)):
        with pytest.raises(ValueError):
            cut(cuda_lib, c, ints([0, 0]), bad, 80, 90)
    with pytest.raises(ValueError):
        cut(cuda_lib, c, None, ints([0, 0]), 80, 90)
