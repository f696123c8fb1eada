"""Pools whose rows lie past 2^32 bytes: keys, block attention, masses and eviction on
pages at a pool's far end, against the same on a small pool."""
import pytest
import torch

from paged_util import DEV, gen, ints

pytestmark = pytest.mark.gpu
SCALE = 512 ** -0.5
P, FAR = 64, 2 ** 32 // 1024 // 64 + 40                  # pages: 4 GB of rows and a few more


def pools(n_pages, base, seed=0):
    """Rows and keys of 40 pages from page `base` of a pool on; the others are not written."""
    g = gen(seed)
    rows = torch.empty(n_pages, P, 512, dtype=torch.bfloat16, device=DEV)
    keys = torch.empty(n_pages, P, 128, dtype=torch.bfloat16, device=DEV)
    rows[base:base + 40] = torch.randn(40, P, 512, generator=g, device=DEV).to(torch.bfloat16)
    keys[base:base + 40] = torch.randn(40, P, 128, generator=g, device=DEV).to(torch.bfloat16)
    return rows, keys


def run(lib, n_pages, base):
    rows, ik = pools(n_pages, base)
    table = (torch.arange(20, device=DEV).view(2, 10) * 7 % 20 + base).to(torch.int32).contiguous()
    n_rows = ints([640, 577])
    keys, n_blocks = torch.zeros(n_pages, 128, dtype=torch.bfloat16, device=DEV), ints([0, 0])
    lib.ds4a_paged_block_keys(ik, table, n_rows, keys, n_blocks)
    g = gen(1)
    iq, w = torch.randn(2, 1, 64, 128, generator=g, device=DEV).to(torch.bfloat16), torch.rand(2, 1, 64, generator=g, device=DEV)
    scores = torch.zeros(2, 1, 10, device=DEV)
    lib.ds4a_paged_block_score(iq, w, keys, table, n_blocks, scores)
    idx, count = ints([[9, 0, 4], [9, 8, 2]]), ints([3, 3])
    q = torch.randn(2, 64, 512, generator=g, device=DEV).to(torch.bfloat16)
    raw, n_raw = torch.randn(2, 128, 512, generator=g, device=DEV).to(torch.float16), ints([128, 3])
    out, lse = torch.zeros(2, 64, 512, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 64, device=DEV)
    ws = torch.empty(lib.ds4a_workspace_bytes(lib.DS4A_OP_PAGED_ATTN_BLOCKS, 2, 1, 3 * P, 0), dtype=torch.uint8, device=DEV)
    lib.ds4a_paged_attn_blocks(q, rows, table, n_rows, idx, count, raw, n_raw, SCALE, out, lse, ws)
    mass = torch.zeros(1, 2, 640, device=DEV)
    lib.ds4a_paged_attn_mass(q, rows, table, n_rows, SCALE, lse, mass, idx=idx, count=count, blocks=True)
    kept = mass.clone()
    free, head = (torch.arange(20, 40, device=DEV) + base).to(torch.int32), ints([6])
    ws = torch.empty(lib.ds4a_workspace_bytes(lib.DS4A_OP_PAGED_EVICT, 2, 1, 640, 200), dtype=torch.uint8, device=DEV)
    lib.ds4a_paged_evict(mass, n_rows, table, rows, free, head, 200, 600, mass, n_rows, table, free, head, ws, recent=20, ik=ik)
    assert n_rows.tolist() == [200, 577] and head.item() == 0
    at = table[0, :4].long()
    return [keys[base:base + 20], scores, out, lse, kept, mass, rows[at].view(-1, 512)[:200], ik[at].view(-1, 128)[:200],
            table[:, :4] - base, free[:10] - base]


def test_far_pages(cuda_lib):
    near = run(cuda_lib, 40, 0)
    # (ten pages come back in front of a head of 6 + 4: none is dropped)
    assert cuda_lib.ds4a_get_device_status() == (0, 0)
    far = run(cuda_lib, FAR, FAR - 40)
    assert cuda_lib.ds4a_get_device_status() == (0, 0)
    for a, b in zip(near, far):
        assert torch.equal(a, b)
