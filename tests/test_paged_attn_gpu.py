"""ds4a_paged_attn_decode against softmax attention in 64 bits over the rows that
the block tables name (bounds: paged_util.check_attn)."""
import random

import pytest
import torch

from paged_util import (DEV, WINDOW, attn_reference, check_attn, e4m3_rows, gen, ints, make_table, pages_of, pool_rows)

pytestmark = pytest.mark.gpu
SCALE = 512 ** -0.5


class Batch:
    """A paged batch; every place that no listed row lies in holds NaN."""

    def __init__(self, lengths, P, H=64, fp8=False, top_k=0, n_raw=None, seed=0, pad=0, spread=1.0, max_pages=None, ring=True):
        g, U = gen(seed), len(lengths)
        self.P, self.H, self.fp8, self.U, self.top_k, self.lengths = P, H, fp8, U, top_k, lengths
        mp = max_pages or max(1, pages_of(max(lengths), P))
        self.table, self.n_pages, _ = make_table(lengths, P, mp, seed=seed, pad=pad)
        used = torch.zeros(self.n_pages * P, dtype=torch.bool, device=DEV)
        for u, n in enumerate(lengths):
            used[pool_rows(self.table, u, torch.arange(n, device=DEV), P)] = True
        vals = torch.randn(self.n_pages * P, 512, generator=g, device=DEV)
        self.row_scale = None
        if fp8:
            codes = (vals * 100).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            codes[~used] = 0x7F
            self.rows = codes.view(self.n_pages, P, 512)
            self.row_scale = torch.exp2(torch.randint(-9, -5, (self.n_pages, P), generator=g, device=DEV).float())
            self.exact = e4m3_rows(codes, self.row_scale.view(-1))
        else:
            rows = vals.to(torch.bfloat16)
            rows[~used] = float("nan")
            self.rows, self.exact = rows.view(self.n_pages, P, 512), rows.double()
        self.q = (torch.randn(U, H, 512, generator=g, device=DEV) * spread).to(torch.bfloat16)
        n_ring = U + 3
        self.raw = torch.randn(n_ring, WINDOW, 512, generator=g, device=DEV).to(torch.float16)
        self.ring = torch.randperm(n_ring, generator=g, device=DEV)[:U].to(torch.int32) if ring else None
        n_raw = [WINDOW] * U if n_raw is None else n_raw
        for u, n in enumerate(n_raw):
            self.raw[int(self.ring[u]) if ring else u, max(0, n):] = float("nan")
        self.n_rows, self.n_raw = ints(lengths), ints(n_raw)
        self.idx = self.count = None
        if top_k:
            self.idx = torch.full((U, top_k), -1, dtype=torch.int32, device=DEV)
            rng, counts = random.Random(seed), []
            for u, n in enumerate(lengths):
                pick = sorted(rng.sample(range(n), min(n, top_k)))
                self.idx[u, :len(pick)] = ints(pick)
                counts.append(len(pick))
            self.count = ints(counts)
        self.out = torch.full((U + 2, H, 512), 7.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((U + 2, H), 7.0, device=DEV)

    def workspace(self, lib):
        flag = lib.DS4A_OP_FLAG_128_HEADS if self.H == 128 else 0
        n = lib.ds4a_workspace_bytes(lib.DS4A_OP_PAGED_ATTN_DECODE | flag, self.U, 1, self.table.shape[1] * self.P, self.top_k)
        return torch.full((n + 64,), 0x7F, dtype=torch.uint8, device=DEV) if n else None

    def __call__(self, lib, scale=SCALE, ws=None, stream=None):
        ws = self.workspace(lib) if ws is None else ws
        lib.ds4a_paged_attn_decode(self.q, self.rows, self.table, self.n_rows, self.raw, self.n_raw, scale,
                                   self.out[1:-1], self.lse[1:-1], ws, idx=self.idx, count=self.count,
                                   row_scale=self.row_scale, ring=self.ring, stream=stream)
        return ws

    def check(self, scale=SCALE, units=None, listed=None):
        for u in range(self.U) if units is None else units:
            n = self.lengths[u]
            if listed is not None and u in listed:
                rows = listed[u]
            elif self.idx is not None:
                rows = self.idx[u, :int(self.count[u])]
            else:
                rows = torch.arange(n, device=DEV)
            nr = min(max(int(self.n_raw[u]), 0), WINDOW)
            ring = u if self.ring is None else int(self.ring[u])
            x = torch.cat((self.exact[pool_rows(self.table, u, rows, self.P)],
                           self.raw[ring, :nr].double() if 0 <= ring < self.raw.shape[0] else self.exact[:0]))
            ref = attn_reference(self.q[u], x, scale)
            check_attn(self.out[1 + u], self.lse[1 + u], *ref)
        assert (self.out[[0, -1]] == 7).all() and (self.lse[[0, -1]] == 7).all()


EDGES = [0, 1, 7, 8, 9, 63, 64, 65, 127, 128, 129, 200, 511, 512, 513]


@pytest.mark.parametrize("H", [64, 128])
@pytest.mark.parametrize("P", [8, 16, 32, 64, 128, 4096])
def test_all_rows(cuda_lib, P, H):
    raw = [0, 1, 63, 64, 65, 127, 128] * 3
    b = Batch(EDGES, P, H, n_raw=raw[:len(EDGES)], pad=3, seed=P)
    b(cuda_lib)
    assert cuda_lib.ds4a_get_device_status() == (0, 0)
    b.check()


@pytest.mark.parametrize("H,P", [(64, 16), (128, 64)])
def test_all_rows_fp8(cuda_lib, H, P):
    b = Batch(EDGES, P, H, fp8=True, n_raw=[128, 0, 65] * 5)
    b(cuda_lib)
    assert cuda_lib.ds4a_get_device_status() == (0, 0)
    b.check()


@pytest.mark.parametrize("H,P", [(64, 16), (128, 64)])
def test_fp8_scales_of_any_size(cuda_lib, H, P):
    """Scales that are no powers of two, and rows of scale 0: logit 0, nothing added but their weight."""
    b = Batch(EDGES, P, H, fp8=True, n_raw=[128, 0, 65] * 5, seed=2)
    b.row_scale *= torch.rand(b.row_scale.shape, generator=gen(5), device=DEV) + 1
    b.row_scale.view(-1)[::7] = 0
    b.exact = e4m3_rows(b.rows.view(-1, 512), b.row_scale.view(-1))
    b(cuda_lib)
    assert cuda_lib.ds4a_get_device_status() == (0, 0)
    b.check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("top_k", [1, 63, 64, 100, 512, 2048])
@pytest.mark.parametrize("H,P", [(64, 64), (128, 8)])
def test_listed_rows(cuda_lib, H, P, top_k, fp8):
    b = Batch([0, 1, 50, 64, 3000, 777, 2], P, H, fp8=fp8, top_k=top_k, n_raw=[0, 128, 5, 64, 128, 0, 100], seed=top_k)
    b(cuda_lib)
    assert cuda_lib.ds4a_get_device_status() == (0, 0)
    b.check()


@pytest.mark.parametrize("H", [64, 128])
def test_one_long_unit_in_many_pieces(cuda_lib, H):
    b = Batch([16384 + 17], 64, H, n_raw=[128])
    b(cuda_lib)
    b.check()


@pytest.mark.parametrize("top_k", [0, 64])
def test_many_ragged_units(cuda_lib, top_k):
    """More units than CTAs, most of them empty or short, one long."""
    rng = random.Random(5)
    lengths = [rng.choice((0, 0, 1, 64, rng.randint(0, 700))) for _ in range(700)]
    lengths[311] = 9000
    raw = [rng.choice((0, 128, rng.randint(0, 128))) for _ in lengths]
    b = Batch(lengths, 32, n_raw=raw, top_k=top_k)
    b(cuda_lib)
    assert cuda_lib.ds4a_get_device_status() == (0, 0)
    b.check(units=list(range(0, 700, 3)) + [311])


@pytest.mark.parametrize("U", [1, 5])
def test_no_row_at_all(cuda_lib, U):
    b = Batch([0] * U, 64, n_raw=[0] * U)
    b(cuda_lib)
    assert cuda_lib.ds4a_get_device_status() == (0, 0)
    assert (b.out[1:-1] == 0).all() and torch.isneginf(b.lse[1:-1]).all()
    b.check()


@pytest.mark.parametrize("scale,spread", [(0.0, 1.0), (-SCALE, 1.0), (SCALE, 12.0), (SCALE, 1e-3)])
def test_scales(cuda_lib, scale, spread):
    b = Batch([300, 64, 5], 64, n_raw=[128, 0, 7], spread=spread)
    b(cuda_lib, scale=scale)
    b.check(scale=scale)


def test_without_rings_and_shared_pages(cuda_lib):
    """Unit u reads ring u; three sequences share their first pages."""
    b = Batch([500, 300, 420], 64, ring=False)
    b.table[1, :4] = b.table[0, :4]
    b.table[2, :4] = b.table[0, :4]
    b(cuda_lib)
    assert cuda_lib.ds4a_get_device_status() == (0, 0)
    b.check()


def flagged(lib):
    return lib.ds4a_get_device_status() == (lib.DS4A_EDEVICE, lib.DS4A_DEV_BOUNDS)


@pytest.mark.parametrize("P", [8, 32, 64, 128])
@pytest.mark.parametrize("bad", [-1, "end", 2 ** 31 - 1])
def test_pages_outside_the_pool(cuda_lib, P, bad):
    """Rows of such a page are masked (a whole tile, part of one, a partial tile) and flagged."""
    b = Batch([400, 130, 64], P)
    wrong = {0: 1, 1: pages_of(130, P) - 1}
    for u, i in wrong.items():
        b.table[u, i] = b.n_pages if bad == "end" else bad
    b(cuda_lib)
    assert flagged(cuda_lib)
    listed = {u: torch.tensor([r for r in range(b.lengths[u]) if r // P != i], device=DEV) for u, i in wrong.items()}
    b.check(listed=listed)


def test_listed_rows_that_do_not_exist(cuda_lib):
    b = Batch([200, 90, 300], 16, top_k=100)
    b.idx[0, 3], b.idx[0, 70], b.idx[2, 0] = -5, 200, 2 ** 31 - 1
    b(cuda_lib)
    assert flagged(cuda_lib)
    listed = {u: torch.tensor([r for r in b.idx[u, :int(b.count[u])].tolist() if 0 <= r < b.lengths[u]], device=DEV)
              for u in (0, 2)}
    b.check(listed=listed)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lengths", [[700, 700, 700], [16384], [5, 60] * 100])
def test_nan_in_a_row_or_a_head_stays(cuda_lib, lengths, fp8):
    """A NaN in a row that counts makes its unit NaN, in one piece or in many, and a NaN in a head's query that head."""
    b = Batch(lengths, 64, fp8=fp8, seed=4)
    row = int(pool_rows(b.table, 0, torch.tensor([lengths[0] // 2], device=DEV), 64)[0])
    keep = b.rows.view(-1, 512)[row].clone()
    b.rows.view(-1, 512)[row, 7] = 0x7F if fp8 else float("nan")
    b(cuda_lib)
    assert torch.isnan(b.out[1].float()).all() and torch.isnan(b.lse[1]).all()
    b.check(units=range(1, min(b.U, 20)))
    b.rows.view(-1, 512)[row] = keep
    b.q[0, 9, 100] = float("nan")
    b(cuda_lib)
    nan = torch.zeros(64, dtype=torch.bool, device=DEV)
    nan[9] = True
    assert torch.equal(torch.isnan(b.out[1].float()).all(-1), nan) and torch.equal(torch.isnan(b.out[1].float()).any(-1), nan)
    assert torch.equal(torch.isnan(b.lse[1]), nan)
    b.check(units=range(1, min(b.U, 20)))
    assert cuda_lib.ds4a_get_device_status() == (0, 0)


def test_lengths_out_of_range(cuda_lib):
    """Clamped and flagged: no length reads outside its table, list or ring."""
    b = Batch([128, 128, 128, 128], 64, top_k=32)
    b.n_rows[0], b.count[1], b.n_raw[2], b.ring[3] = -3, 99, 4000, b.raw.shape[0]
    b(cuda_lib)
    assert flagged(cuda_lib)
    b.check(listed={0: torch.arange(0, device=DEV), 1: b.idx[1], 2: b.idx[2]})
    b = Batch([128], 64)
    b.n_rows[0] = 2 ** 30                         # its table names 128 rows
    b(cuda_lib)
    assert flagged(cuda_lib)
    b.check()


def test_far_pool_rows(cuda_lib):
    """Rows past 2^32 bytes (and 2^31 elements) of the pool."""
    P, n_pages = 4096, 1200                       # 5.03 GB of rows
    rows = torch.zeros(n_pages, P, 512, dtype=torch.bfloat16, device=DEV)
    b = Batch([700, 64], P, n_raw=[128, 0])
    far = [n_pages - 1, n_pages - 2]
    for u in (0, 1):
        rows[far[u]] = b.rows[int(b.table[u, 0])]
        b.table[u, 0] = far[u]
    b.rows, b.n_pages = rows, n_pages
    for top_k in (0, 40):
        if top_k:
            b.top_k, b.idx, b.count = 40, ints([list(range(1, 400, 10)), list(range(0, 40))]), ints([40, 40])
        b(cuda_lib)
        assert cuda_lib.ds4a_get_device_status() == (0, 0)
        b.exact = rows.view(-1, 512)[-2 * P:].double()
        b.table -= n_pages - 2                    # the reference sees the last two pages alone
        b.check()
        b.table += n_pages - 2


def test_same_result_twice_and_in_other_company(cuda_lib):
    """Bit-identical from call to call, and with one workspace for two batches."""
    b, c = Batch([3000, 0, 65], 64, seed=1), Batch([100, 2048], 64, seed=2)
    ws = max(b.workspace(cuda_lib), c.workspace(cuda_lib), key=lambda t: t.numel())
    b(cuda_lib, ws=ws)
    first = b.out.clone(), b.lse.clone()
    for _ in range(3):
        c(cuda_lib, ws=ws)
        b(cuda_lib, ws=ws)
        assert torch.equal(b.out, first[0]) and torch.equal(b.lse, first[1])
    c.check()


def test_two_streams(cuda_lib):
    b, c = Batch([5000] * 4, 64, seed=1), Batch([900] * 40, 16, seed=2)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    keep = [(b(cuda_lib, stream=s), c(cuda_lib, stream=t)) for _ in range(5)]
    torch.cuda.synchronize()
    del keep
    b.check()
    c.check(units=[0, 17, 39])


def test_captured_batch(cuda_lib):
    """A captured call replayed on a batch with other lengths, pages and padding units."""
    P, mp = 64, 16
    b = Batch([1000, 900, 400, 64], P, max_pages=mp, seed=1)
    ws = b(cuda_lib)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b(cuda_lib, ws=ws)
    for lengths, raw in (([5, 900, 0, 1000], [5, 128, 0, 128]), ([0] * 4, [0] * 4), ([64, 0, 0, 0], [128, 0, 0, 0])):
        c = Batch(lengths, P, max_pages=mp, seed=sum(lengths), n_raw=raw)
        n = min(c.rows.shape[0], b.rows.shape[0])
        assert n == c.rows.shape[0]
        b.rows[:n].copy_(c.rows)
        for k in ("q", "raw", "ring", "n_rows", "n_raw", "table"):
            getattr(b, k).copy_(getattr(c, k))
        graph.replay()
        c.out, c.lse = b.out, b.lse
        c.check()


def test_without_lse(cuda_lib):
    b = Batch([700, 3], 64)
    cuda_lib.ds4a_paged_attn_decode(b.q, b.rows, b.table, b.n_rows, b.raw, b.n_raw, SCALE, b.out[1:-1], None,
                                    b.workspace(cuda_lib), ring=b.ring)
    b.lse[1:-1] = torch.stack([attn_reference(b.q[u], torch.cat((
        b.exact[pool_rows(b.table, u, torch.arange(n, device=DEV), 64)], b.raw[int(b.ring[u])].double())), SCALE)[1]
        for u, n in enumerate(b.lengths)]).float()
    b.check()


def test_rejects_other_tensors(cuda_lib):
    b = Batch([100, 64], 64, top_k=16)
    ws = b.workspace(cuda_lib)
    good = dict(q=b.q, rows=b.rows, table=b.table, n_rows=b.n_rows, raw=b.raw, n_raw=b.n_raw, scale=SCALE, out=b.out[1:-1],
                lse=b.lse[1:-1], ws=ws, idx=b.idx, count=b.count, ring=b.ring)
    for change in (dict(q=b.q.float()), dict(q=b.q.cpu()), dict(q=b.q.transpose(0, 1)), dict(rows=b.rows.half()),
                   dict(rows=b.rows[:, :, :256]), dict(rows=b.rows.view(torch.uint8)[:, :, :512]), dict(table=b.table.long()),
                   dict(table=b.table[:1]), dict(n_rows=b.n_rows[:1]), dict(raw=b.raw.bfloat16()), dict(raw=b.raw[:, :64]),
                   dict(n_raw=b.n_raw.long()), dict(out=b.out[1:-1].float()), dict(out=b.out), dict(lse=b.lse), dict(idx=None),
                   dict(count=None), dict(idx=b.idx[:, ::2]), dict(ring=b.ring[:1]), dict(ring=None, raw=b.raw[:1]),
                   dict(ws=ws.cpu())):
        with pytest.raises(ValueError):
            cuda_lib.ds4a_paged_attn_decode(**dict(good, **change))
    for change in (dict(ws=None), dict(ws=ws[:64]), dict(scale=float("nan")), dict(q=b.q[:, :32].contiguous(),
                                                                                 out=b.out[1:-1, :32].contiguous(), lse=None)):
        with pytest.raises(cuda_lib.Ds4aError):
            cuda_lib.ds4a_paged_attn_decode(**dict(good, **change))
