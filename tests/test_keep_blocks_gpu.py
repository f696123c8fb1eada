"""A list of just the kept blocks: the first and the newest, whatever the others score."""
import pytest
import torch

from paged_util import DEV, gen, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first,last", [(2, 1), (0, 3), (3, 0), (1, 2)])
@pytest.mark.parametrize("U,NB", [(3, 40), (700, 130)])
def test_kept_blocks_fill_the_list(cuda_lib, U, NB, first, last):
    g = gen(U + first)
    n = [NB - u % 5 if u % 3 else u % 7 for u in range(U)]
    table = torch.arange(NB, dtype=torch.int32, device=DEV).repeat(U, 1)
    keys = torch.randn(NB, 128, generator=g, device=DEV).to(torch.bfloat16)
    iq = torch.randn(U, 1, 64, 128, generator=g, device=DEV).to(torch.bfloat16)
    w = torch.rand(U, 1, 64, generator=g, device=DEV)
    scores = torch.full((U, 1, NB), float("nan"), device=DEV)
    cuda_lib.ds4a_paged_block_score(iq, w, keys, table, ints(n), scores, first, last)
    k = first + last
    idx, count = (torch.empty(U, 1, m, dtype=torch.int32, device=DEV) for m in (k, 1))
    cuda_lib.ds4a_topk_select(scores, ints(n), k, idx, count.view(U, 1), None)
    assert cuda_lib.ds4a_get_device_status() == (0, 0)
    for u in range(U):
        want = sorted(set(range(min(first, n[u]))) | set(range(max(n[u] - last, 0), n[u])))
        got = idx[u, 0, :int(count[u])].tolist()
        assert len(got) == min(k, n[u]) and set(want) <= set(got)
