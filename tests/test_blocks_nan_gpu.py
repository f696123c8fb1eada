"""A key that is not a number makes its page's score NaN, which no list holds; the other
pages' scores, and those selected whatever they score, are not touched by it."""
import pytest
import torch

from paged_util import DEV, gen, ints

pytestmark = pytest.mark.gpu
P = 8


@pytest.mark.parametrize("U,NB", [(3, 300), (200, 400)])          # a block a tile, and the scan of large batches
@pytest.mark.parametrize("where", ["key", "rows", "iq", "w"])
def test_nan(cuda_lib, U, NB, where):
    g = gen(U)
    n = [NB - u % 9 for u in range(U)]
    table = torch.randperm(U * NB, generator=g, device=DEV).to(torch.int32).view(U, NB)
    ik = torch.randn(U * NB, P, 128, generator=g, device=DEV).to(torch.bfloat16)
    iq = torch.randn(U, 1, 64, 128, generator=g, device=DEV).to(torch.bfloat16)
    w = torch.rand(U, 1, 64, generator=g, device=DEV)
    keys, n_blocks = torch.zeros(U * NB, 128, dtype=torch.bfloat16, device=DEV), ints(n)

    def score():
        got = torch.full((U, 1, NB), 77.0, device=DEV)
        cuda_lib.ds4a_paged_block_score(iq, w, keys, table, n_blocks, got, 1, 2)
        return got[:, 0]

    def fill():
        cuda_lib.ds4a_paged_block_keys(ik, table, ints([m * P for m in n]), keys, torch.empty_like(n_blocks))
    fill()
    clean = score()
    bad = torch.zeros(U, NB, dtype=torch.bool, device=DEV)
    if where in ("key", "rows"):
        for u, b in ((0, 5), (0, 131), (1, 0), (2, 299 - 10), (U - 1, 7), (U - 1, n[U - 1] - 1)):
            bad[u, b] = True
        pages = table[bad].long()
        if where == "key":
            keys[pages, 77] = float("nan")
        else:
            ik[pages, 3, 0] = float("nan")
            fill()
            assert keys[pages, 0].isnan().all() and not keys[pages, 1:].isnan().any()
    elif where == "iq":
        iq[1, 0, 63, 127] = float("nan")
        bad[1] = True
    else:
        w[1, 0, 40] = float("nan")
        bad[1] = True
    got = score()
    assert cuda_lib.ds4a_get_device_status() == (0, 0)
    i = torch.arange(NB, device=DEV)[None, :]
    there, kept = i < n_blocks[:, None], (i < 1) | (i >= n_blocks[:, None] - 2)
    assert got[bad & there & ~kept].isnan().all() and (bad & there & ~kept).any()
    assert torch.isposinf(got[there & kept]).all()
    same = ~(bad & there & ~kept)
    assert torch.equal(got[same], clean[same])
    # none of them is selected, however long the list
    idx, count = torch.empty(U, 1, NB, dtype=torch.int32, device=DEV), torch.empty(U, 1, dtype=torch.int32, device=DEV)
    cuda_lib.ds4a_topk_select(got.view(U, 1, NB).contiguous(), n_blocks, NB, idx, count, None)
    assert cuda_lib.ds4a_get_device_status() == (0, 0)
    want = there & (kept | ~bad)
    for u in sorted({0, 1, 2, U - 1}):
        assert idx[u, 0, :int(count[u])].tolist() == want[u].nonzero().flatten().tolist()


def test_infinite_keys(cuda_lib):
    """max(0, -inf) is 0 and max(0, inf) infinite, as the formula has it."""
    table, keys = torch.arange(4, dtype=torch.int32, device=DEV)[None], torch.zeros(4, 128, dtype=torch.bfloat16, device=DEV)
    iq = torch.ones(1, 1, 64, 128, dtype=torch.bfloat16, device=DEV)
    w, got = torch.ones(1, 1, 64, device=DEV), torch.empty(1, 1, 4, device=DEV)
    keys[0], keys[1, 0], keys[2, 0] = 1.0, float("inf"), -float("inf")
    keys[3, 0], keys[3, 1] = float("inf"), -float("inf")
    cuda_lib.ds4a_paged_block_score(iq, w, keys, table, ints([4]), got)
    assert cuda_lib.ds4a_get_device_status() == (0, 0)
    s = got.flatten().tolist()
    assert s[0] == 64 * 128 and s[1] == float("inf") and s[2] == 0 and s[3] != s[3]
