"""ds4a_paged_plan against a walk over the sequences (whole numbers: equal)."""
import random

import pytest
import torch

from paged_util import DEV, gen, ints, pages_of, plan_reference

pytestmark = pytest.mark.gpu
KEYS = ("n_rows", "n_raw", "cu_tok", "cu_row", "tok_pos", "raw_slot", "row_pos", "row_slot")


class Plan:
    """One step's inputs and outputs on the device, with room around every output."""

    def __init__(self, past, add, ratio, P, extra=5, ring=True, head=3, pad=2, seed=0, T_cap=None, R_cap=None, free=None,
                 max_pages=None, off=0):
        self.past, self.add, self.ratio, self.P, self.head = past, add, ratio, P, head
        B = len(past)
        rng = random.Random(seed)
        held = [pages_of(p // ratio, P) for p in past]
        want = [pages_of((p + a) // ratio, P) for p, a in zip(past, add)]
        n = sum(want) + head + 4
        pages = torch.randperm(n, generator=gen(seed, "cpu")).tolist()
        at = sum(held)
        self.max_pages = max_pages or max(1, max(want))
        self.table, k = [], 0
        for h in held:
            self.table.append(pages[k:k + h] + [-9] * (self.max_pages - h))
            k += h
        self.free = pages[at:] if free is None else free
        self.ring = rng.sample(range(B + 5), B) if ring else None
        self.T_cap = sum(add) + extra if T_cap is None else T_cap
        self.R_cap = max(1, sum((p + a) // ratio - p // ratio for p, a in zip(past, add)) + extra) if R_cap is None else R_cap
        self.T_cap = max(1, self.T_cap)
        self.d_table = torch.full((B, self.max_pages + pad), -9, dtype=torch.int32, device=DEV)
        self.d_table[:, :self.max_pages] = ints(self.table)
        self.room, self.out = {}, {}
        for name, size in dict(n_rows=B, n_raw=B, cu_tok=B + 1, cu_row=B + 1, tok_pos=self.T_cap, raw_slot=self.T_cap,
                               row_pos=self.R_cap, row_slot=self.R_cap).items():
            room = torch.full((size + 8 + off,), -77, dtype=torch.int32, device=DEV)
            self.room[name], self.out[name] = room, room[4 + off:4 + off + size]
        self.off = off
        self.d_head, self.d_head_out = ints([head]), ints([-77])
        self.d_free, self.d_past, self.d_add = ints(self.free), ints(past), ints(add)
        self.d_ring = ints(self.ring) if ring else None

    def __call__(self, lib, head_out=None):
        o = self.out
        lib.ds4a_paged_plan(self.d_past, self.d_add, self.ratio, self.P, self.d_free, self.d_head,
                            self.d_table[:, :self.max_pages], o["n_rows"], o["n_raw"], o["cu_tok"], o["cu_row"],
                            o["tok_pos"], o["raw_slot"], o["row_pos"], o["row_slot"],
                            self.d_head_out if head_out is None else head_out, ring=self.d_ring)

    def check(self):
        want, table, head = plan_reference(self.past, self.add, self.ratio, self.P, self.free, self.head, self.table,
                                           self.ring, self.T_cap, self.R_cap)
        for k in KEYS:
            assert self.out[k].tolist() == want[k], k
            assert (self.room[k][:4 + self.off] == -77).all() and (self.room[k][-4:] == -77).all(), k
        assert self.d_table[:, :self.max_pages].tolist() == table
        assert (self.d_table[:, self.max_pages:] == -9).all()
        return head


def status(lib):
    return lib.ds4a_get_device_status()


@pytest.mark.parametrize("B", [1, 2, 33, 1025, 8192])
@pytest.mark.parametrize("ratio,P", [(4, 64), (128, 8), (1, 4096), (3, 16)])
def test_decode_steps(cuda_lib, B, ratio, P):
    rng = random.Random(B * 1000 + ratio)
    past = [rng.randint(0, 4000) for _ in range(B)]
    p = Plan(past, [1] * B, ratio, P, seed=B)
    p(cuda_lib)
    assert status(cuda_lib) == (0, 0)
    assert p.d_head_out.item() == p.check()


@pytest.mark.parametrize("off", [0, 1])          # outputs off a 16-byte boundary take the scalar stores
@pytest.mark.parametrize("seed,ratio,P", [(0, 4, 64), (1, 128, 8), (2, 4, 8), (3, 2, 256)])
def test_prompt_chunks(cuda_lib, seed, ratio, P, off):
    rng = random.Random(seed)
    B = 61
    past = [rng.choice((0, rng.randint(0, 3), rng.randint(0, 5000))) for _ in range(B)]
    add = [rng.choice((0, 1, 127, 128, 129, rng.randint(0, 2048))) for _ in range(B)]
    add[0], add[-1] = 0, 0                        # nothing new at both ends
    p = Plan(past, add, ratio, P, ring=bool(seed % 2), seed=seed, off=off)
    p(cuda_lib)
    assert status(cuda_lib) == (0, 0)
    assert p.d_head_out.item() == p.check()


def test_nothing_new(cuda_lib):
    p = Plan([0, 7, 0], [0, 0, 0], 4, 64)
    p(cuda_lib)
    assert status(cuda_lib) == (0, 0) and p.d_head_out.item() == p.check()


def test_far_positions(cuda_lib):
    top = 2 ** 31 - 1
    p = Plan([top - 300], [300], 2 ** 20, 4096)
    p(cuda_lib)
    assert status(cuda_lib) == (0, 0) and p.d_head_out.item() == p.check()


@pytest.mark.parametrize("add", [1, 2048])        # one CTA, and a cluster
def test_head_in_place_and_steps_in_a_row(cuda_lib, add):
    """Steps behind one another on one stream, the free list's head updated in
    place and the lengths advanced on the device."""
    B, ratio, P = 9, 4, 8
    first = Plan([5 * b for b in range(B)], [3 * add] * B, ratio, P, max_pages=4000 if add > 1 else 20)
    past, table, head = first.past, first.table, first.head
    first.d_add.fill_(add)
    steps = []
    for _ in range(3):
        o = {k: torch.empty_like(v) for k, v in first.out.items()}
        cuda_lib.ds4a_paged_plan(first.d_past, first.d_add, ratio, P, first.d_free, first.d_head,
                                 first.d_table[:, :first.max_pages], *[o[k] for k in KEYS], first.d_head, ring=first.d_ring)
        first.d_past += first.d_add
        steps.append(o)
    for o in steps:
        want, table, head = plan_reference(past, [add] * B, ratio, P, first.free, head, table, first.ring, first.T_cap,
                                           first.R_cap)
        for k in KEYS:
            assert o[k].tolist() == want[k], k
        past = [p + add for p in past]
    assert first.d_table[:, :first.max_pages].tolist() == table and first.d_head.item() == head
    assert status(cuda_lib) == (0, 0)


def test_free_list_runs_out(cuda_lib):
    p = Plan([0, 0, 0], [64, 64, 64], 4, 8, head=1, free=[50, 51, 52, 53])      # six pages wanted, three there
    p(cuda_lib)
    assert status(cuda_lib) == (cuda_lib.DS4A_EDEVICE, cuda_lib.DS4A_DEV_BOUNDS)
    assert p.d_head_out.item() == 4
    assert p.d_table[:, :2].tolist() == [[51, 52], [53, -1], [-1, -1]]
    rows = [pg * 8 + r if pg >= 0 else -1 for pg in (51, 52, 53, -1, -1, -1) for r in range(8)]
    assert p.out["row_slot"].tolist() == rows + [-1] * 5
    assert p.out["n_rows"].tolist() == [16, 16, 16]


def test_sequence_outgrows_its_table(cuda_lib):
    p = Plan([0, 0], [64, 32], 4, 8, max_pages=1)
    p.d_table.fill_(-9)
    p(cuda_lib)
    assert status(cuda_lib) == (cuda_lib.DS4A_EDEVICE, cuda_lib.DS4A_DEV_BOUNDS)
    f = p.free[p.head:]
    assert p.d_table[:, 0].tolist() == [f[0], f[2]] and (p.d_table[:, 1:] == -9).all()
    assert p.out["row_slot"].tolist() == [f[0] * 8 + r for r in range(8)] + [-1] * 8 + [f[2] * 8 + r for r in range(8)] + [-1] * 5


def test_capacities_too_small(cuda_lib):
    full = Plan([3, 9], [40, 30], 4, 8)
    want, _, _ = plan_reference(full.past, full.add, 4, 8, full.free, full.head, full.table, full.ring, full.T_cap, full.R_cap)
    p = Plan([3, 9], [40, 30], 4, 8, T_cap=50, R_cap=6)
    p(cuda_lib)
    assert status(cuda_lib) == (cuda_lib.DS4A_EDEVICE, cuda_lib.DS4A_DEV_BOUNDS)
    for k, n in (("tok_pos", 50), ("raw_slot", 50), ("row_pos", 6), ("row_slot", 6)):
        assert p.out[k].tolist() == want[k][:n]
        assert (p.room[k][-4:] == -77).all()
    assert p.out["cu_tok"].tolist() == want["cu_tok"]


def test_bad_lengths_and_rings(cuda_lib):
    p = Plan([8, 8, 8, 8], [4, 4, 4, 4], 4, 8, extra=0)
    p.d_past[1] = -5
    p.d_add[2] = -1
    p.d_past[3] = 2 ** 31 - 4
    p.d_add[3] = 4                                 # past the last position: no new token
    p.d_ring[0] = -2
    p.d_table[:, :p.max_pages] = 7
    p(cuda_lib)
    assert status(cuda_lib) == (cuda_lib.DS4A_EDEVICE, cuda_lib.DS4A_DEV_BOUNDS)
    assert p.out["cu_tok"].tolist() == [0, 4, 8, 8, 8]
    assert p.out["tok_pos"].tolist() == [8, 9, 10, 11, 0, 1, 2, 3] + [-1] * 8
    assert p.out["raw_slot"].tolist()[:4] == [-1] * 4
    assert p.out["raw_slot"].tolist()[4:8] == [p.ring[1] * 128 + i for i in range(4)]
    assert p.out["n_rows"].tolist() == [3, 1, 2, (2 ** 31 - 4) // 4]


def test_rejects_other_tensors(cuda_lib):
    p = Plan([8, 8], [4, 4], 4, 8)
    good = p.d_past
    for bad in (good.long(), good.cpu(), torch.stack((good, good), 1)[:, 0], good[:1]):
        p.d_past = bad
        with pytest.raises(ValueError):
            p(cuda_lib)


def test_captured_step(cuda_lib):
    """A captured step replayed on other lengths, its arrays behind the last token -1."""
    p = Plan([0] * 7, [40] * 7, 4, 8, extra=0)
    p(cuda_lib)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p(cuda_lib)
    for past, add in (([3] * 7, [2] * 7), ([0] * 7, [0, 5, 0, 9, 40, 1, 0])):
        q = Plan(past, add, 4, 8, T_cap=p.T_cap, R_cap=p.R_cap, max_pages=p.max_pages)
        p.d_past.copy_(q.d_past), p.d_add.copy_(q.d_add), p.d_table.copy_(q.d_table)
        p.d_ring.copy_(q.d_ring), p.d_free[:len(q.free)].copy_(q.d_free[:p.d_free.numel()])
        graph.replay()
        want, table, head = plan_reference(past, add, 4, 8, p.d_free.tolist(), p.head, q.table, q.ring, p.T_cap, p.R_cap)
        for k in KEYS:
            assert p.out[k].tolist() == want[k], k
        assert p.d_table[:, :p.max_pages].tolist() == table and p.d_head_out.item() == head
