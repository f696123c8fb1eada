"""Eviction with a workspace that holds anything: what the copies go by is what the select
of the same call wrote."""
import pytest
import torch

from paged_util import DEV, ints
from test_evict_gpu import Cache, status

pytestmark = pytest.mark.gpu


def call(lib, c, ws, keep, limit, **kw):
    """The eviction of Cache.run, out of place, with this workspace."""
    c.before = {k: None if getattr(c, k) is None else getattr(c, k).clone()
                for k in ("rows", "row_scale", "ik", "mass", "table", "free_pages", "n_rows", "gone")}
    c.first_row = torch.full((c.B,), -9, dtype=torch.int32, device=DEV)
    c.out = {k: torch.full_like(getattr(c, k), 77) for k in ("mass", "n_rows", "free_pages", "free_head", "gone")}
    c.out["table"] = torch.full((c.B, c.table.stride(0)), 77, dtype=torch.int32, device=DEV)[:, :c.max_pages]
    lib.ds4a_paged_evict(c.mass, c.n_rows, c.table, c.rows, c.free_pages, c.free_head, keep, limit, c.out["mass"],
                         c.out["n_rows"], c.out["table"], c.out["free_pages"], c.out["free_head"], ws, row_scale=c.row_scale,
                         ik=c.ik, gone=c.gone, gone_out=c.out["gone"], first_row=c.first_row, **kw)
    c.in_place, c.sizes = False, (keep, limit, kw.get("first", 0), kw.get("recent", 0), [0] * c.B)


@pytest.mark.parametrize("fill", [0x00, 0x01, 0x7F, 0xFF])
def test_evict_with_a_workspace_of_anything(cuda_lib, fill):
    """Every word set before the call, and then another batch over what the first one left."""
    need = cuda_lib.ds4a_workspace_bytes(cuda_lib.DS4A_OP_PAGED_EVICT, 8192, 1, 64, 20)
    ws = torch.full((need,), fill, dtype=torch.uint8, device=DEV)
    for lengths, max_pages, keep, limit, kw in (([5, 60, 33, 64, 0] * 1638 + [40, 64], 8, 20, 32, dict(first=2, recent=5)),
                                                ([300, 0, 101, 64], 40, 100, 100, {}),
                                                ([0, 9, 40], 8, 40, 64, {})):
        c = Cache(lengths, 8, 1, max_pages=max_pages, ik=False)
        call(cuda_lib, c, ws, keep, limit, **kw)
        status(cuda_lib)
        c.check()


def test_evict_refused_over_a_workspace_of_another_batch(cuda_lib):
    """No sequence is cut: nothing of the batch before comes back."""
    ws = torch.empty(1 << 16, dtype=torch.uint8, device=DEV)
    call(cuda_lib, Cache([500, 400, 300], 16), ws, 200, 250)
    status(cuda_lib)
    c = Cache([500, 400, 300], 16, seed=1)
    c.free_head.fill_(-1)
    c.head = -1
    call(cuda_lib, c, ws, 200, 250)
    status(cuda_lib, True)
    c.check(refused=(0, 1, 2))
    c = Cache([500, 400, 300], 16, seed=2)
    c.n_rows.copy_(ints([100, 250, 0]))
    c.lengths = [100, 250, 0]
    call(cuda_lib, c, ws, 200, 250)
    status(cuda_lib)
    c.check()
