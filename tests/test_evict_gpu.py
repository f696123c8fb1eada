"""Accumulated attention weights against the formula in 64 bits, eviction against a
walk in Python, and plans after evictions."""
import math
import random
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

from paged_util import DEV, e4m3_rows, gen, ints, make_table, pages_of, plan_reference, pool_rows

pytestmark = pytest.mark.gpu
SCALE = 512 ** -0.5


def status(lib, bad=False):
    assert lib.ds4a_get_device_status() == ((lib.DS4A_EDEVICE, lib.DS4A_DEV_BOUNDS) if bad else (0, 0))


# ------------------------------------------------------------------------------------------ mass
class Mass:
    def __init__(self, lengths, P, H=64, kind="all", lists=None, fp8=False, seed=0, top_k=None, extra=0):
        g, U = gen(seed), len(lengths)
        self.lengths, self.P, self.H, self.U, self.kind, self.lists = lengths, P, H, U, kind, lists
        self.table, self.n_pages, _ = make_table(lengths, P, max(1, pages_of(max(lengths), P)), seed=seed)
        nan = 0x7F if fp8 else float("nan")
        pool = torch.full((self.n_pages * P, 512), nan, dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEV)
        for u, n in enumerate(lengths):
            x = torch.randn(n, 512, generator=g, device=DEV)
            at = pool_rows(self.table, u, torch.arange(n, device=DEV), P)
            pool[at] = (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else x.to(torch.bfloat16)
        self.rows = pool.view(self.n_pages, P, 512)
        self.row_scale = torch.exp2(torch.randint(-9, -5, (self.n_pages, P), generator=g, device=DEV).float()) if fp8 else None
        self.q = torch.randn(U, H, 512, generator=g, device=DEV).to(torch.bfloat16)
        self.idx = self.count = None
        if lists is not None:
            k = top_k or max(1, max(len(x) for x in lists))
            idx = torch.full((U, k), -1, dtype=torch.int32)
            for u, x in enumerate(lists):
                idx[u, :len(x)] = torch.tensor(x, dtype=torch.int32)
            self.idx, self.count = idx.to(DEV), ints([len(x) for x in lists])
        self.n_rows = ints(lengths)
        # about what an attention over the rows and a window gives
        self.lse = torch.log(self.n_rows.float() + 128)[:, None] + 0.5 + 0.3 * torch.randn(U, H, generator=g, device=DEV)
        self.start = torch.rand(H // 64, U, self.table.shape[1] * P + extra, generator=g, device=DEV)
        self.mass = self.start.clone()

    def __call__(self, lib, **kw):
        lib.ds4a_paged_attn_mass(self.q, self.rows, self.table, self.n_rows, SCALE, self.lse, self.mass, idx=self.idx,
                                 count=self.count, blocks=self.kind == "blocks", row_scale=self.row_scale, **kw)

    def rows_of(self, u):
        if self.kind == "all":
            return list(range(self.lengths[u]))
        if self.kind == "rows":
            return self.lists[u]
        return [b * self.P + i for b in self.lists[u] for i in range(self.P) if b * self.P + i < self.lengths[u]]

    def check(self, times=1, units=None, skip=()):
        """A logit is a sum of 512 exact products in fp32 (e, as an attention's), scaled and
        shifted by -lse in log2 units (2^-22 of either); 2^x is off by 2^-21, and 64
        weights and the old mass are added in fp32."""
        for u in range(self.U) if units is None else units:
            r = [] if u in skip else self.rows_of(u)
            want, tol = self.start[:, u].double(), torch.zeros_like(self.start[:, u], dtype=torch.float64)
            if r:
                at = torch.tensor(r, device=DEV)
                p = pool_rows(self.table, u, at, self.P)
                x = self.rows.view(-1, 512)[p]
                x = x.double() if self.row_scale is None else e4m3_rows(x, self.row_scale.view(-1)[p])
                q, lse = self.q[u].double(), self.lse[u].double()
                z = q @ x.T * SCALE
                e = 512 * 2.0 ** -24 * (q.abs() @ x.abs().T) * SCALE + 2.0 ** -22 * (z.abs() + lse.abs()[:, None])
                w = torch.exp(z - lse[:, None])
                rel = torch.expm1(e) + 2.0 ** -21 + 64 * 2.0 ** -24
                want = want.clone()
                for _ in range(times):
                    want.index_add_(1, at, w.view(-1, 64, len(r)).sum(1))
                    tol.index_add_(1, at, (w * rel).view(-1, 64, len(r)).sum(1))
            tol = tol + 4 * times * 2.0 ** -24 * want.abs()
            assert ((self.mass[:, u].double() - want).abs() <= tol).all()
            rest = torch.ones(self.mass.shape[2], dtype=torch.bool, device=DEV)
            if r:
                rest[torch.tensor(r, device=DEV)] = False
            assert torch.equal(self.mass[:, u, rest], self.start[:, u, rest])


LENGTHS = [0, 1, 8, 47, 48, 49, 100, 257, 513, 1000]


@pytest.mark.parametrize("P", [8, 16, 64, 256])
@pytest.mark.parametrize("H,fp8", [(64, False), (128, False), (64, True), (128, True)])
@pytest.mark.parametrize("kind", ["all", "rows", "blocks"])
def test_mass(cuda_lib, P, H, fp8, kind):
    rng = random.Random(P)
    lists = None
    if kind != "all":
        most = [n if kind == "rows" else pages_of(n, P) for n in LENGTHS]
        lists = [rng.sample(range(n), min(n, 60 if kind == "rows" else 5)) for n in most]
    m = Mass(LENGTHS, P, H, kind, lists, fp8, seed=P, extra=5, top_k=70 if lists else None)
    m(cuda_lib)
    status(cuda_lib)
    m.check()


def test_mass_is_the_attentions_own(cuda_lib):
    """With the attention's lse the rows' masses and the window's weights sum to one a head."""
    m = Mass([700, 90, 0, 1], 16)
    raw, n_raw = torch.randn(4, 128, 512, generator=gen(1), device=DEV).to(torch.float16), ints([0, 0, 0, 0])
    out = torch.empty(4, 64, 512, dtype=torch.bfloat16, device=DEV)
    n = cuda_lib.ds4a_workspace_bytes(cuda_lib.DS4A_OP_PAGED_ATTN_DECODE, 4, 1, m.table.shape[1] * 16, 0)
    cuda_lib.ds4a_paged_attn_decode(m.q, m.rows, m.table, m.n_rows, raw, n_raw, SCALE, out, m.lse,
                                    torch.empty(n, dtype=torch.uint8, device=DEV))
    assert torch.isneginf(m.lse[2]).all()
    m.mass.zero_()
    m.start.zero_()
    m(cuda_lib)
    status(cuda_lib)
    assert (m.mass[0].sum(1) - torch.tensor([64.0, 64.0, 0.0, 64.0], device=DEV)).abs().max() < 64 * 1e-4
    m.lse[2] = 0
    m.check()


def test_mass_of_a_batch_twice_and_the_same_bits(cuda_lib):
    rng = random.Random(2)
    lengths = [rng.choice((0, 1, rng.randint(0, 4000))) for _ in range(300)]
    m = Mass(lengths, 64)
    m(cuda_lib)
    first = m.mass.clone()
    m.check(units=range(0, 300, 13))
    m(cuda_lib)
    m.check(times=2, units=range(0, 300, 29))
    m.mass.copy_(m.start)
    m(cuda_lib)
    assert torch.equal(m.mass, first)


@pytest.mark.parametrize("kind", ["rows", "blocks"])
def test_mass_of_entries_listed_twice(cuda_lib, kind):
    lists = [[3, 3, 1], [5, 2, 5, 5]] if kind == "blocks" else [[3] * 100 + [700], list(range(90)) * 2]
    m = Mass([800, 400], 64, 128, kind, lists)
    m(cuda_lib)
    status(cuda_lib)
    for u in range(2):
        r = torch.tensor(m.rows_of(u), device=DEV)
        p = pool_rows(m.table, u, r, 64)
        z = m.q[u].double() @ m.rows.view(-1, 512)[p].double().T * SCALE
        w = torch.exp(z - m.lse[u].double()[:, None]).view(2, 64, -1).sum(1)
        want = m.start[:, u].double().index_add_(1, r, w)
        assert ((m.mass[:, u].double() - want).abs() <= 2.0 ** -13 * want).all()
    first = m.mass.clone()
    for _ in range(3):
        m.mass.copy_(m.start)
        m(cuda_lib)
        assert torch.equal(m.mass, first)


def test_mass_of_units_without_a_token(cuda_lib):
    m = Mass([500, 300, 0, 64], 16)
    m(cuda_lib, tok_pos=ints([-1, 0, 5, -1]))
    status(cuda_lib)
    m.check(skip=(0, 3))


def test_mass_out_of_range(cuda_lib):
    m = Mass([300, 300], 16, kind="rows", lists=[[1, 299, 5], [0, 7]], top_k=4)
    m.idx[0, 1] = 300
    m.idx[1, 0] = -1
    m(cuda_lib)
    status(cuda_lib, True)
    m.lists = [[1, 5], [7]]
    m.check()
    m = Mass([300, 300], 16)
    m.n_rows.copy_(ints([-1, 5000]))
    m.lengths = [0, 304]
    m.rows.copy_(torch.randn_like(m.rows))
    m(cuda_lib)
    status(cuda_lib, True)
    m.check()
    m = Mass([300, 300], 16)
    m.table[0, 2] = m.n_pages
    m(cuda_lib)
    status(cuda_lib, True)
    keep = [r for r in range(300) if r // 16 != 2]
    m.kind, m.lists, m.table[0, 2] = "rows", [keep, list(range(300))], 0
    m.check()


def test_mass_of_special_lse(cuda_lib):
    m = Mass([100], 16)
    m.lse[0, 3] = -math.inf
    m.lse[0, 4] = math.inf
    m(cuda_lib)
    z = m.q[0].double() @ m.rows.view(-1, 512)[pool_rows(m.table, 0, torch.arange(100, device=DEV), 16)].double().T * SCALE
    w = torch.exp(z - m.lse[0].double()[:, None])
    w[3] = 0
    want = m.start[0, 0].double()
    want[:100] += w.sum(0)
    assert ((m.mass[0, 0].double() - want).abs() <= 2.0 ** -13 * want).all()
    m.lse[0, 5] = float("nan")
    m(cuda_lib)
    assert m.mass[0, 0, :100].isnan().all()


def test_mass_captured_and_on_two_streams(cuda_lib):
    a, b = Mass([3000, 10, 900], 32, 128), Mass([2000] * 60, 64, kind="rows", lists=[list(range(5, 500))] * 60, seed=4)
    a(cuda_lib), b(cuda_lib)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a(cuda_lib)
    a.mass.copy_(a.start), b.mass.copy_(b.start)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graph.replay()
    b(cuda_lib, stream=t)
    torch.cuda.synchronize()
    a.check(), b.check(units=[0, 31, 59])


# ----------------------------------------------------------------------------------------- evict
class Cache:
    """A paged cache of B sequences; every row and key holds numbers of its own."""

    def __init__(self, lengths, P, planes=1, fp8=False, ik=True, seed=0, n_free=None, max_pages=None, mass=None, used=3):
        g, B = gen(seed), len(lengths)
        self.lengths, self.P, self.B, self.fp8 = lengths, P, B, fp8
        self.max_pages = max_pages or max(1, pages_of(max(lengths), P))
        held = sum(pages_of(n, P) for n in lengths)
        spare = held + 5 if n_free is None else n_free
        self.table, self.n_pages, free = make_table(lengths, P, self.max_pages, spare=spare, seed=seed, pad=1)
        # `used` entries of the list were taken by others, then the pages that these sequences hold
        self.head = used + held
        taken = [int(self.table[u, i]) for u, n in enumerate(lengths) for i in range(pages_of(n, P))]
        self.free = [7] * used + taken + free
        self.rows = torch.randint(0, 120 if fp8 else 2 ** 15, (self.n_pages, P, 512), generator=g, device=DEV)
        self.rows = self.rows.to(torch.uint8) if fp8 else self.rows.to(torch.int16).view(torch.bfloat16)
        self.row_scale = torch.rand(self.n_pages, P, generator=g, device=DEV) if fp8 else None
        self.ik = torch.randn(self.n_pages, P, 128, generator=g, device=DEV).to(torch.bfloat16) if ik else None
        self.mass = torch.rand(planes, B, self.max_pages * P + 2, generator=g, device=DEV) if mass is None else mass
        self.n_rows, self.free_pages, self.free_head = ints(lengths), ints(self.free), ints([self.head])
        self.gone = ints([3 * b for b in range(B)])

    def bits(self, t):
        return None if t is None else t.view(torch.uint8 if self.fp8 and t.dtype == torch.uint8 else
                                             torch.int32 if t.dtype == torch.float32 else torch.int16)

    def run(self, lib, keep, limit, first=0, recent=0, in_place=True, n_shared=None, stream=None):
        self.before = {k: None if getattr(self, k) is None else getattr(self, k).clone()
                       for k in ("rows", "row_scale", "ik", "mass", "table", "free_pages", "n_rows", "gone")}
        ws = torch.empty(lib.ds4a_workspace_bytes(lib.DS4A_OP_PAGED_EVICT, self.B, 1, self.max_pages * self.P, keep),
                         dtype=torch.uint8, device=DEV)
        self.first_row = torch.full((self.B,), -9, dtype=torch.int32, device=DEV)
        names = ("mass", "n_rows", "table", "free_pages", "free_head", "gone")
        out = {k: getattr(self, k) for k in names}
        if not in_place:
            out = {k: torch.full_like(v, 77) for k, v in out.items()}
            full = torch.full((self.B, self.table.stride(0)), 77, dtype=torch.int32, device=DEV)
            out["table"] = full[:, :self.max_pages]
        self.call = lambda: lib.ds4a_paged_evict(
            self.mass, self.n_rows, self.table, self.rows, self.free_pages, self.free_head, keep, limit, out["mass"],
            out["n_rows"], out["table"], out["free_pages"], out["free_head"], ws, first=first, recent=recent,
            row_scale=self.row_scale, ik=self.ik, gone=self.gone, gone_out=out["gone"], first_row=self.first_row,
            n_shared=None if n_shared is None else ints(n_shared), stream=stream)
        torch.cuda.synchronize()
        self.call()
        self.out, self.in_place = out, in_place
        self.sizes = (keep, limit, first, recent, n_shared or [0] * self.B)

    def check(self, refused=()):
        keep, limit, first, recent, n_shared = self.sizes
        b4, P, need = self.before, self.P, pages_of(keep, self.P)
        table = b4["table"].tolist()
        mass = b4["mass"].sum(0) if b4["mass"].shape[0] <= 2 else None
        if mass is None:
            mass = b4["mass"][0].clone()
            for p in range(1, b4["mass"].shape[0]):
                mass = mass + b4["mass"][p]
        mass = mass.tolist()
        head, back, evicted = self.head, [], {}
        for b, n in enumerate(self.lengths):
            if n <= limit or b in refused:
                continue
            middle = range(first, n - recent)
            rank = sorted(middle, key=lambda r: (1, 0.0, r) if math.isnan(mass[b][r]) else (0, -mass[b][r], r))
            kept = sorted(list(range(first)) + rank[:keep - first - recent] + list(range(n - recent, n)))
            evicted[b] = (kept, self.free[head:head + need])
            head += need
            back += table[b][n_shared[b]:pages_of(n, P)]
        head -= len(back)
        o = self.out
        assert o["free_head"].item() == head
        want_free = b4["free_pages"].tolist() if self.in_place else [77] * len(self.free)
        want_free[head:head + len(back)] = back
        assert o["free_pages"].tolist() == want_free
        assert o["n_rows"].tolist() == [keep if b in evicted else n for b, n in enumerate(b4["n_rows"].tolist())]
        assert o["gone"].tolist() == [x + (self.lengths[b] - keep if b in evicted else 0) for b, x in enumerate(b4["gone"].tolist())]
        assert self.first_row.tolist() == [0 if b in evicted else max(n, 0) for b, n in enumerate(b4["n_rows"].tolist())]
        want_table = b4["table"].tolist() if self.in_place else [[77] * self.max_pages for _ in range(self.B)]
        want_mass = b4["mass"].clone() if self.in_place else torch.full_like(self.mass, 77)
        want = {k: None if b4[k] is None else b4[k].clone() for k in ("rows", "row_scale", "ik")}
        for b, (kept, pages) in evicted.items():
            want_table[b][:need] = pages
            at = torch.tensor(kept, device=DEV)
            want_mass[:, b, :self.lengths[b]] = 0
            want_mass[:, b, :keep] = b4["mass"][:, b, at]
            src = pool_rows(b4["table"], b, at, P)
            j = torch.arange(keep, device=DEV)
            dst = torch.tensor(pages, device=DEV)[j // P] * P + j % P
            for k, v in want.items():
                if v is not None:
                    v.view(self.n_pages * P, -1)[dst] = b4[k].view(self.n_pages * P, -1)[src]
        assert o["table"].tolist() == want_table
        assert torch.equal(o["mass"].nan_to_num(-5), want_mass.nan_to_num(-5))
        for k, v in want.items():
            if v is not None:
                got, ref = self.bits(getattr(self, k)).view(self.n_pages, P, -1), self.bits(v).view(self.n_pages, P, -1)
                # (the last new page's rows behind the kept ones hold anything)
                for b, (kept, pages) in evicted.items():
                    if keep % P:
                        got[pages[-1], keep % P:] = ref[pages[-1], keep % P:]
                assert torch.equal(got, ref), k


@pytest.mark.parametrize("P", [8, 16, 64, 256])
@pytest.mark.parametrize("planes,fp8,ik,in_place", [(1, False, True, True), (2, True, False, False), (2, False, False, True),
                                                    (3, True, True, False)])
def test_evict(cuda_lib, P, planes, fp8, ik, in_place):
    c = Cache([0, 1, 99, 100, 101, 120, 121, 300, 1000, 64, 777], P, planes, fp8, ik, seed=P)
    c.run(cuda_lib, 100, 120, first=4, recent=10, in_place=in_place)
    status(cuda_lib)
    c.check()


@pytest.mark.parametrize("keep,limit,first,recent", [(1, 1, 0, 0), (1, 1, 1, 0), (1, 5, 0, 1), (64, 64, 0, 64), (64, 64, 64, 0),
                                                     (63, 64, 30, 33), (65, 70, 0, 0), (512, 600, 4, 100), (1000, 1000, 0, 1)])
def test_evict_sizes(cuda_lib, keep, limit, first, recent):
    c = Cache([1001, 64, 65, 2, 0, 5000], 32, 2, seed=keep)
    c.run(cuda_lib, keep, limit, first, recent)
    status(cuda_lib)
    c.check()


def test_evict_ties_zeros_and_nans(cuda_lib):
    n = [700, 700, 700, 700, 700]
    mass = torch.zeros(2, 5, 704 + 64, device=DEV)
    mass[0, 1] = torch.randint(0, 4, (768,), generator=gen(1), device=DEV).float()
    mass[1, 1] = torch.randint(0, 4, (768,), generator=gen(2), device=DEV).float()
    mass[0, 2] = torch.rand(768, generator=gen(3), device=DEV)
    mass[0, 2, ::3] = float("nan")
    mass[0, 3, :] = -torch.rand(768, generator=gen(4), device=DEV)          # (no attention gives these)
    mass[0, 3, 50:60] = math.inf
    mass[1, 3, 55:70] = -math.inf
    mass[0, 4] = float("nan")
    c = Cache(n, 64, 2, mass=mass)
    c.run(cuda_lib, 300, 400, 5, 20)
    status(cuda_lib)
    c.check()


def test_evict_long_sequences(cuda_lib):
    """Past the keys that fit into shared memory, and just within."""
    for n, keep, max_pages in ((60000, 9000, None), (20000, 16000, 768), (49152, 30001, 768)):
        c = Cache([n, 500, n - 777], 64, 1, True, False, seed=1, max_pages=max_pages)
        c.run(cuda_lib, keep, keep, 4, 1000)
        status(cuda_lib)
        c.check()


def test_evict_a_large_batch(cuda_lib):
    rng = random.Random(7)
    c = Cache([rng.choice((0, rng.randint(0, 40), rng.randint(0, 90))) for _ in range(1500)], 8, 1, True)
    c.run(cuda_lib, 30, 50, 2, 5)
    status(cuda_lib)
    c.check()


def test_evict_the_largest_batch(cuda_lib):
    """8,192 sequences, more of them over the limit than there are SMs, and hardly any."""
    rng = random.Random(8)
    for share in (0.1, 0.001):
        lengths = [rng.randint(33, 64) if rng.random() < share else rng.randint(0, 32) for _ in range(8192)]
        c = Cache(lengths, 8, 1, True, False, max_pages=8)
        c.run(cuda_lib, 20, 32, 2, 5)
        status(cuda_lib)
        c.check()


def test_evict_nothing(cuda_lib):
    for lengths in ([0], [100, 64, 0]):
        c = Cache(lengths, 16, max_pages=8)
        c.run(cuda_lib, 100, 100)
        status(cuda_lib)
        c.check()


def test_evict_with_shared_pages(cuda_lib):
    c = Cache([500, 300, 40, 500], 16, n_free=200)
    c.table[3, :20] = c.table[0, :20]                # the first 20 pages are held by both (its own are nobody's)
    c.run(cuda_lib, 200, 250, 0, 16, n_shared=[20, 100, 0, 20])
    status(cuda_lib)
    c.check()


def test_evict_with_a_short_free_list(cuda_lib):
    c = Cache([500, 100, 400, 450, 300], 16, n_free=2 * 13 + 12)     # three want 13 pages each, two get them
    c.run(cuda_lib, 200, 310)
    status(cuda_lib, True)
    c.check(refused=(3,))
    c = Cache([500, 100], 16)
    c.free_head.fill_(-1)
    c.head = -1
    c.run(cuda_lib, 200, 310)
    status(cuda_lib, True)
    c.check(refused=(0,))


def test_evict_out_of_range(cuda_lib):
    c = Cache([500, 100, 400], 16)
    c.n_rows[1] = -4                                 # clamped to 0, left as it is
    c.run(cuda_lib, 200, 310)
    status(cuda_lib, True)
    c.check()
    c = Cache([500, 100, 400], 16)
    c.n_rows[0] = 10 ** 9                            # clamped to the table's rows
    c.lengths[0] = c.max_pages * 16
    c.run(cuda_lib, 200, 310)
    status(cuda_lib, True)
    b4 = c.before["n_rows"].clone()
    c.before["n_rows"][0] = 512
    c.check()
    assert int(b4[0]) == 10 ** 9
    for where in ("old", "new"):                     # a page that is not one of the pool's: left as it is, its new pages lost
        c = Cache([500, 100, 400], 16)
        if where == "old":
            c.table[0, 7] = c.n_pages
        else:
            c.free_pages[c.head + 3] = -1
        rows, table = c.rows.clone(), c.table.clone()
        c.run(cuda_lib, 200, 310)
        status(cuda_lib, True)
        assert c.out["n_rows"].tolist() == [500, 100, 200] and torch.equal(c.table[:2], table[:2])
        assert c.free_head.item() == c.head + 2 * 13 - 25
        assert c.table[2, :13].tolist() == c.free[c.head + 13:c.head + 26]
        assert torch.equal(rows.view(torch.int16)[table[0, :7].long()], c.rows.view(torch.int16)[table[0, :7].long()])


def test_evict_drops_pages_past_the_lists_start(cuda_lib):
    c = Cache([500], 16, used=0)
    c.free_pages = ints([900 + i for i in range(5)] + c.free[c.head:])       # a list that never held the old pages
    c.free, c.head = c.free_pages.tolist(), 5
    c.free_head.fill_(5)
    c.run(cuda_lib, 200, 310)
    status(cuda_lib, True)
    assert c.free_head.item() == 0                   # 5 + 13 - 32 is below the start: the last 18 fit
    assert c.free_pages.tolist()[:18] == c.before["table"][0, 14:32].tolist()
    assert c.n_rows.tolist() == [200]


def test_evict_captured_and_on_another_stream(cuda_lib):
    c = Cache([500, 100, 400, 320], 16, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.run(cuda_lib, 200, 310, 4, 16, in_place=False, stream=s)
    s.synchronize()
    c.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.call()
    for lengths in ([500, 90, 311, 0], [310, 20, 0, 5], [499, 100, 400, 311]):
        c.lengths = lengths
        c.n_rows.copy_(ints(c.lengths))
        for k in ("mass", "n_rows", "table", "free_pages", "free_head", "gone"):
            c.out[k].fill_(77)
        c.before = {k: None if getattr(c, k) is None else getattr(c, k).clone()
                    for k in ("rows", "row_scale", "ik", "mass", "table", "free_pages", "n_rows", "gone")}
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        status(cuda_lib)
        c.check()


def in_two_threads(*calls):
    """Each call many times over, in a thread of its own and on a stream of its own."""
    def many(call):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(2000):
                call()
    torch.cuda.synchronize()
    with ThreadPoolExecutor(len(calls)) as pool:
        for done in [pool.submit(many, call) for call in calls]:
            done.result()
    torch.cuda.synchronize()


@pytest.mark.parametrize("lengths", [([40000], [500, 100]), ([9] * 8192, [5, 9] * 2700)])
def test_evict_in_two_threads(cuda_lib, lengths):
    """Calls of different sizes, whose kernels need different amounts of shared memory."""
    caches = [Cache(n, 8, seed=k) for k, n in enumerate(lengths)]
    for c in caches:
        c.run(cuda_lib, 8, 8, in_place=False)
    in_two_threads(*(c.call for c in caches))
    status(cuda_lib)
    for c in caches:
        c.check()


# ------------------------------------------------------------------------------ plans afterwards
def test_plan_in_two_threads(cuda_lib):
    def plan(B):
        table = torch.full((B, 2), -1, dtype=torch.int32, device=DEV)
        table[:, 0] = torch.arange(B, device=DEV)
        o = [torch.zeros(n, dtype=torch.int32, device=DEV) for n in (B, B, B + 1, B + 1, 4 * B, 4 * B, B, B, 1)]
        args = (ints([40] * B), ints([4] * B), 4, 8, ints(list(range(B, 3 * B))), ints([0]), table, *o)
        return o, lambda: cuda_lib.ds4a_paged_plan(*args, gone=gone[B])
    gone = {B: ints([5] * B) for B in (8192, 2000)}
    plans = {B: plan(B) for B in gone}
    in_two_threads(*(call for _, call in plans.values()))
    status(cuda_lib)
    for B, (o, _) in plans.items():
        assert o[0].tolist() == [6] * B and o[8].item() == 0


@pytest.mark.parametrize("form", [0, 1, 3, 4, 7])
@pytest.mark.parametrize("ratio,P", [(4, 8), (1, 64), (128, 16)])
def test_plan_after_evictions(cuda_lib, form, ratio, P):
    """The plan of the rows held, with positions that count the evicted ones."""
    rng = random.Random(form * 100 + ratio)
    B = 40
    by_seq = form & 3
    past = [rng.choice((0, rng.randint(0, 3000))) for _ in range(B)]
    add = [rng.randint(0, 1) if by_seq else rng.choice((0, 1, rng.randint(0, 500))) for _ in range(B)]
    gone = [rng.choice((0, rng.randint(0, p // ratio), p // ratio)) for p in past]
    held = [p - g * ratio for p, g in zip(past, gone)]
    cap = max(pages_of((h + a) // ratio, P) for h, a in zip(held, add)) + 1
    table, n_pages, _ = make_table([h // ratio for h in held], P, cap, spare=900)
    free, head = list(range(n_pages - 900, n_pages)), 4
    T, R = max(sum(add) + 3, B), max(sum(add) + 3, B)
    o = {k: torch.full((n,), -7, dtype=torch.int32, device=DEV)
         for k, n in (("n_rows", B), ("n_raw", B), ("cu_tok", B + 1), ("cu_row", B + 1), ("tok_pos", T), ("raw_slot", T),
                      ("row_pos", R), ("row_slot", R), ("head", 1))}
    want, want_table, want_head = plan_reference(held, add, ratio, P, free, head, table.tolist(), None, T, R)
    cuda_lib.ds4a_paged_plan(ints(past), ints(add), ratio, P, ints(free), ints([head]), table, o["n_rows"], o["n_raw"],
                             o["cu_tok"], o["cu_row"], o["tok_pos"], o["raw_slot"], o["row_pos"], o["row_slot"], o["head"],
                             form=form, gone=ints(gone))
    status(cuda_lib)
    assert table.tolist() == want_table and o["head"].item() == want_head
    for k in ("n_rows", "cu_tok", "cu_row"):
        assert o[k].tolist() == want[k], k
    assert o["n_raw"].tolist() == [min(p + a, 128) for p, a in zip(past, add)]
    tok, row = [], []
    for b in range(B):
        end = past[b] + add[b]
        new = [(pos, b * 128 + pos % 128 if pos >= end - 128 else -1) for pos in range(past[b], end)]
        tok += (new or [(-1, -1)]) if form & 1 else new
        first = 0 if form & 4 else ratio - 1
        at = want["row_slot"][want["cu_row"][b]:want["cu_row"][b + 1]]
        new = [(j * ratio + first, s) for j, s in zip(range(past[b] // ratio, end // ratio), at)]
        row += (new or [(-1, -1)]) if form & 2 else new
    for (p, s), got, n in ((("tok_pos", "raw_slot"), tok, T), (("row_pos", "row_slot"), row, R)):
        got += [(-1, -1)] * (n - len(got))
        assert o[p].tolist() == [x for x, _ in got] and o[s].tolist() == [y for _, y in got]


@pytest.mark.parametrize("form,most", [(0, 3), (0, 70), (3, 1)])
def test_plan_of_the_largest_batch(cuda_lib, form, most):
    """8,192 sequences, most of them never cut: the plan of the tokens that are left, on one
    block, every SM and by sequence."""
    rng = random.Random(9)
    B, ratio, P = 8192, 4, 8
    past, add = [rng.randint(0, 200) for _ in range(B)], [rng.randint(0, most) for _ in range(B)]
    gone = [rng.choice((0, 0, p // ratio)) for p in past]
    T = max(sum(add), B)

    def plan(past, **kw):
        table = torch.full((B, 9), -1, dtype=torch.int32, device=DEV)
        table[:, :8] = torch.arange(B * 8, device=DEV).view(B, 8)
        o = [torch.zeros(n, dtype=torch.int32, device=DEV) for n in (B, B, B + 1, B + 1, T, T, T, T, 1)]
        cuda_lib.ds4a_paged_plan(ints(past), ints(add), ratio, P, ints(list(range(B * 8, B * 24))), ints([0]), table, *o,
                                 form=form, **kw)
        status(cuda_lib)
        return table, o
    table, o = plan(past, gone=ints(gone))
    held = [p - g * ratio for p, g in zip(past, gone)]
    want_table, want = plan(held)
    assert torch.equal(table, want_table)
    for k in (0, 2, 3, 7, 8):                        # n_rows, cu_tok, cu_row, row_slot, head: by the rows held
        assert torch.equal(o[k], want[k]), k
    same = plan(past)[1]
    assert torch.equal(o[1], same[1]) and torch.equal(o[4], same[4]) and torch.equal(o[5], same[5])
    assert torch.equal(o[6], same[6])                # positions: by the tokens


def test_plan_with_gone_out_of_range(cuda_lib):
    table = torch.full((2, 8), -1, dtype=torch.int32, device=DEV)
    o = [torch.zeros(n, dtype=torch.int32, device=DEV) for n in (2, 2, 3, 3, 4, 4, 4, 4, 1)]
    cuda_lib.ds4a_paged_plan(ints([40, 40]), ints([4, 4]), 4, 8, ints(list(range(16))), ints([0]), table, *o,
                             gone=ints([11, -1]))
    status(cuda_lib, True)
    assert o[0].tolist() == [11, 11]                 # counted as 0


# ------------------------------------------------------------------------------------- refusals
def test_rejects_other_tensors(cuda_lib):
    m = Mass([100, 64], 16)
    good = dict(q=m.q, rows=m.rows, table=m.table, n_rows=m.n_rows, scale=SCALE, lse=m.lse, mass=m.mass)
    for change in (dict(lse=m.lse.double()), dict(lse=m.lse[:1]), dict(mass=m.mass[0]), dict(mass=m.mass.half()),
                   dict(mass=m.mass[:, :1]), dict(mass=m.mass.repeat(2, 1, 1)), dict(idx=m.n_rows), dict(q=m.q.float()),
                   dict(tok_pos=m.n_rows[:1])):
        with pytest.raises(ValueError):
            cuda_lib.ds4a_paged_attn_mass(**dict(good, **change))
    with pytest.raises(cuda_lib.Ds4aError):
        cuda_lib.ds4a_paged_attn_mass(**dict(good, mass=torch.zeros(1, 2, 111, device=DEV)))
    c = Cache([100, 64], 16)
    c.run(cuda_lib, 80, 90)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device=DEV)
    good = dict(mass=c.mass, n_rows=c.n_rows, table=c.table, rows=c.rows, free_pages=c.free_pages, free_head=c.free_head,
                keep=80, limit=90, mass_out=c.mass, n_rows_out=c.n_rows, table_out=c.table, free_pages_out=c.free_pages,
                free_head_out=c.free_head, ws=ws, ik=c.ik)
    for change in (dict(mass=c.mass[0]), dict(mass_out=c.mass[:, :, :-1]), dict(rows=c.rows.float()), dict(ik=c.ik[:1]),
                   dict(table_out=c.table.contiguous()), dict(free_pages_out=c.free_pages[:-1]), dict(n_rows_out=c.n_rows[:1]),
                   dict(gone=c.gone[:1]), dict(ws=ws.cpu()), dict(rows=c.rows.view(torch.uint8)[:, :, :512])):
        with pytest.raises(ValueError):
            cuda_lib.ds4a_paged_evict(**dict(good, **change))
    for change in (dict(keep=0), dict(limit=79), dict(first=50, recent=31), dict(ws=None)):
        with pytest.raises(cuda_lib.Ds4aError):
            cuda_lib.ds4a_paged_evict(**dict(good, **change))
