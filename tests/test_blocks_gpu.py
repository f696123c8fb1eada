"""Block keys, block scores and attention over listed blocks against the formulas in
64 bits, at the lengths, page sizes and lists where they can go wrong."""
import math
import random

import pytest
import torch

from paged_util import DEV, WINDOW, attn_reference, check_attn, e4m3_rows, gen, ints, make_table, pages_of, pool_rows

pytestmark = pytest.mark.gpu
SCALE = 512 ** -0.5
BOUNDS = "BOUNDS"


def status(lib, want=None):
    got = lib.ds4a_get_device_status()
    assert got == ((0, 0) if want is None else (lib.DS4A_EDEVICE, lib.DS4A_DEV_BOUNDS))


# ------------------------------------------------------------------------------------------ keys
class KeyStore:
    def __init__(self, lengths, P, seed=0, pad=0, max_pages=None):
        g = gen(seed)
        self.lengths, self.P = lengths, P
        self.table, self.n_pages, _ = make_table(lengths, P, max_pages or max(1, pages_of(max(lengths), P)), seed=seed, pad=pad)
        keys = torch.full((self.n_pages * P, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
        for u, n in enumerate(lengths):
            keys[pool_rows(self.table, u, torch.arange(n, device=DEV), P)] = \
                torch.randn(n, 128, generator=g, device=DEV).to(torch.bfloat16)
        self.ik = keys.view(self.n_pages, P, 128)
        self.n_rows, self.n_blocks = ints(lengths), torch.full((len(lengths),), -7, dtype=torch.int32, device=DEV)
        self.block_keys = torch.full((self.n_pages, 128), 7.0, dtype=torch.bfloat16, device=DEV)

    def __call__(self, lib, **kw):
        lib.ds4a_paged_block_keys(self.ik, self.table, self.n_rows, self.block_keys, self.n_blocks, **kw)

    def check(self, first):
        """The pages from row first[u] on hold their means, the others 7."""
        done = set()
        assert self.n_blocks.tolist() == [pages_of(n, self.P) for n in self.lengths]
        for u, n in enumerate(self.lengths):
            if first[u] >= n:
                continue
            for b in range(first[u] // self.P, pages_of(n, self.P)):
                page = int(self.table[u, b])
                done.add(page)
                k = self.ik[page, :min(self.P, n - b * self.P)].double()
                ref = k.mean(0)
                # c sums and a division in fp32, one rounding to bf16
                err = (k.shape[0] + 1) * 2.0 ** -24 * k.abs().mean(0)
                assert ((self.block_keys[page].double() - ref).abs() <= err + 2.0 ** -8 * (ref.abs() + err)).all()
        rest = [p for p in range(self.n_pages) if p not in done]
        assert (self.block_keys[rest] == 7).all()


EDGES = [0, 1, 7, 8, 9, 63, 64, 65, 127, 128, 129, 300, 1000]


@pytest.mark.parametrize("P", [8, 16, 32, 64, 128, 256, 1024, 4096])
def test_keys_of_all_rows(cuda_lib, P):
    k = KeyStore(EDGES, P, seed=P, pad=3)
    k(cuda_lib)
    status(cuda_lib)
    k.check([0] * len(EDGES))


@pytest.mark.parametrize("P", [8, 64, 256])
@pytest.mark.parametrize("by", ["cu_row", "first_row"])
def test_keys_of_new_rows(cuda_lib, P, by):
    rng = random.Random(P)
    k = KeyStore(EDGES * 20, P, seed=1)
    new = [rng.choice((0, min(n, 1), rng.randint(0, n), n)) for n in k.lengths]
    first = [n - a for n, a in zip(k.lengths, new)]
    if by == "cu_row":
        cu = torch.cat((ints([0]), torch.cumsum(ints(new), 0).to(torch.int32)))
        k(cuda_lib, cu_row=cu)
    else:
        k(cuda_lib, first_row=ints(first))
    status(cuda_lib)
    k.check(first)


def test_keys_out_of_range(cuda_lib):
    for kw, first in ((dict(first_row=ints([-1, 300])), [0, 300]), (dict(cu_row=ints([0, 200, 100])), [0, 300])):
        k = KeyStore([100, 300], 64)
        k(cuda_lib, **kw)
        status(cuda_lib, BOUNDS)
        k.check(first)
    k = KeyStore([100, 300], 64)                     # a length past the table, and below zero
    k.n_rows.copy_(ints([-5, 1000]))
    k.lengths = [0, 320]
    k.ik.copy_(torch.randn_like(k.ik))
    k(cuda_lib)
    status(cuda_lib, BOUNDS)
    k.check([0, 0])
    k = KeyStore([100, 300], 64)                     # a page that is not one of the pool's is left out
    k.table[1, 2] = k.n_pages
    k(cuda_lib)
    status(cuda_lib, BOUNDS)
    assert k.n_blocks.tolist() == [2, 5]


# ---------------------------------------------------------------------------------------- scores
class Scores:
    def __init__(self, blocks, NB_cap, seed=0, pad=0, max_pages=None):
        g, U = gen(seed), len(blocks)
        self.blocks, self.NB_cap = blocks, NB_cap
        self.table, self.n_pages, unused = make_table(blocks, 1, max_pages or max(1, max(blocks)), seed=seed, pad=pad)
        self.keys = torch.randn(self.n_pages, 128, generator=g, device=DEV).to(torch.bfloat16)
        self.keys[unused] = float("nan")
        self.iq = torch.randn(U, 1, 64, 128, generator=g, device=DEV).to(torch.bfloat16)
        self.w = torch.randn(U, 1, 64, generator=g, device=DEV)
        self.n_blocks = ints(blocks)
        self.scores = torch.full((U, 1, NB_cap), 7.0, device=DEV)

    def __call__(self, lib, **kw):
        lib.ds4a_paged_block_score(self.iq, self.w, self.keys, self.table, self.n_blocks, self.scores, **kw)

    def check(self, n_first=0, n_last=0, units=None, bad=()):
        for u in range(len(self.blocks)) if units is None else units:
            n = self.blocks[u]
            assert (self.scores[u, 0, n:] == 7).all()
            b = torch.arange(n, device=DEV)
            got = self.scores[u, 0, :n]
            out = torch.zeros(n, dtype=torch.bool, device=DEV)
            for x, i in bad:
                if x == u:
                    out[i] = True
            ends = ((b < n_first) | (b >= n - n_last)) & ~out
            assert torch.isposinf(got[ends]).all() and torch.isneginf(got[out]).all()
            rest = ~ends & ~out
            k = self.keys[self.table[u, :n][rest].long()].double()
            q, w = self.iq[u, 0].double(), self.w[u, 0].double()
            ref = ((k @ q.T).relu() * w).sum(-1)
            # 128 products, 64 weighted heads and 2 roundings in fp32
            tol = 194 * 2.0 ** -24 * ((k.abs() @ q.abs().T) * w.abs()).sum(-1) + 1e-30
            assert ((got[rest].double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("n_first,n_last", [(0, 0), (1, 2), (5, 0), (0, 2 ** 31 - 1)])
def test_scores(cuda_lib, n_first, n_last):
    s = Scores([0, 1, 2, 3, 127, 128, 129, 256, 500], 501, pad=2)
    s(cuda_lib, n_first=n_first, n_last=n_last)
    status(cuda_lib)
    s.check(n_first, n_last)


def test_scores_of_many_and_long_units(cuda_lib):
    rng = random.Random(3)
    s = Scores([rng.choice((0, 1, rng.randint(0, 600))) for _ in range(300)], 20000, max_pages=20000)
    s.blocks[17] = 0
    s.n_blocks[17] = 0
    s(cuda_lib)
    status(cuda_lib)
    s.check(units=range(0, 300, 9))
    s = Scores([20000], 20000)
    s(cuda_lib, n_last=1)
    s.check(0, 1)


def test_scores_of_a_batch_of_short_units(cuda_lib):
    """Every tile another unit's: queries change with each."""
    rng = random.Random(4)
    s = Scores([rng.choice((0, 1, 2, 3, 100, 130)) for _ in range(3000)], 130)
    s(cuda_lib, n_first=1, n_last=1)
    status(cuda_lib)
    s.check(1, 1, units=range(0, 3000, 17))


@pytest.mark.parametrize("cap", [300, 60000])        # a block of threads per tile, and the persistent scan
@pytest.mark.parametrize("bad", [-1, "end", 2 ** 31 - 1])
def test_scores_of_pages_outside_the_pool(cuda_lib, bad, cap):
    s = Scores([300, 40], cap, max_pages=cap)
    s.table[0, 130] = s.n_pages if bad == "end" else bad
    s.table[0, 299] = -1                             # a last block too
    s(cuda_lib, n_last=1)
    status(cuda_lib, BOUNDS)
    s.check(0, 1, bad=((0, 130), (0, 299)))


@pytest.mark.parametrize("cap", [100, 60000])
@pytest.mark.parametrize("n,limit", [(-1, 0), ("over", "cap"), (2 ** 31 - 1, "cap")])
def test_block_counts_out_of_range(cuda_lib, n, limit, cap):
    n, limit = cap + 1 if n == "over" else n, cap if limit == "cap" else limit
    s = Scores([cap, 90], cap)
    s.n_blocks[0] = n
    s.blocks[0] = limit
    s(cuda_lib)
    status(cuda_lib, BOUNDS)
    s.check()


def test_captured_keys_scores_and_selection(cuda_lib):
    """Keys, scores and the selection that reads the counts right behind them."""
    P, U, k = 16, 4, 8
    store = KeyStore([900, 1000, 500, 130], P, max_pages=64)
    cu = ints([0, 900, 1900, 2400, 2530])
    s = Scores([1] * U, 64)
    idx, count = torch.empty(U, 1, k, dtype=torch.int32, device=DEV), torch.empty(U, 1, dtype=torch.int32, device=DEV)

    def run():
        store(cuda_lib, cu_row=cu)
        cuda_lib.ds4a_paged_block_score(s.iq, s.w, store.block_keys, store.table, store.n_blocks, s.scores, 1, 1)
        cuda_lib.ds4a_topk_select(s.scores, store.n_blocks, k, idx, count, None)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for lengths in ([900, 1000, 500, 130], [0, 17, 16, 129], [1, 1000, 333, 2]):
        store.lengths = lengths
        store.n_rows.copy_(ints(lengths))
        cu.copy_(torch.cat((ints([0]), torch.cumsum(ints(lengths), 0).to(torch.int32))))
        store.block_keys.fill_(7.0)
        s.scores.fill_(7.0)
        graph.replay()
        status(cuda_lib)
        store.check([0] * U)
        for u, n in enumerate(lengths):
            m = pages_of(n, P)
            want = s.scores[u, 0, :m].sort(descending=True, stable=True).indices[:k].sort().values
            assert int(count[u]) == min(m, k) and idx[u, 0, :min(m, k)].tolist() == want.tolist()
            assert m == 0 or (0 in want.tolist() and (m - 1) in want.tolist())


# ------------------------------------------------------------------------------------- attention
class Attention:
    def __init__(self, lengths, lists, P, H=64, fp8=False, seed=0, top_k=None, n_raw=None, pad=0):
        g, U = gen(seed), len(lengths)
        self.lengths, self.lists, self.P, self.H, self.U = lengths, lists, P, H, U
        self.table, self.n_pages, _ = make_table(lengths, P, max(1, pages_of(max(lengths), P)), seed=seed, pad=pad)
        nan = 0x7F if fp8 else float("nan")
        pool = torch.full((self.n_pages * P, 512), nan, dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEV)
        for u, n in enumerate(lengths):
            x = torch.randn(n, 512, generator=g, device=DEV)
            at = pool_rows(self.table, u, torch.arange(n, device=DEV), P)
            pool[at] = (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else x.to(torch.bfloat16)
        self.rows = pool.view(self.n_pages, P, 512)
        self.row_scale = torch.exp2(torch.randint(-9, -5, (self.n_pages, P), generator=g, device=DEV).float()) if fp8 else None
        self.q = torch.randn(U, H, 512, generator=g, device=DEV).to(torch.bfloat16)
        k = top_k or max(1, max(len(x) for x in lists))
        idx = torch.full((U, k), -1, dtype=torch.int32)
        for u, x in enumerate(lists):
            idx[u, :len(x)] = torch.tensor(x, dtype=torch.int32)
        self.idx, self.count = idx.to(DEV), ints([len(x) for x in lists])
        self.n_rows = ints(lengths)
        self.n_raw = [WINDOW if u % 3 else (u * 37) % 129 for u in range(U)] if n_raw is None else n_raw
        self.raw = torch.randn(U + 1, WINDOW, 512, generator=g, device=DEV).to(torch.float16)
        for u, n in enumerate(self.n_raw):
            self.raw[U - u, n:] = float("nan")
        self.ring = ints([U - u for u in range(U)])
        self.out = torch.full((U, H, 512), 7.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((U, H), 7.0, device=DEV)
        self.raw_n = ints(self.n_raw)
        self.ws = None

    def __call__(self, lib, **kw):
        if self.ws is None:
            op = lib.DS4A_OP_PAGED_ATTN_BLOCKS | (lib.DS4A_OP_FLAG_128_HEADS if self.H == 128 else 0)
            n = lib.ds4a_workspace_bytes(op, self.U, 1, self.idx.shape[1] * self.P, 0)
            self.ws = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
        lib.ds4a_paged_attn_blocks(self.q, self.rows, self.table, self.n_rows, self.idx, self.count, self.raw, self.raw_n, SCALE,
                                   self.out, self.lse, self.ws, row_scale=self.row_scale, ring=self.ring, **kw)

    def values(self, u, skip=()):
        r = [b * self.P + i for b in self.lists[u] if b not in skip for i in range(self.P)]
        r = torch.tensor([x for x in r if x < self.lengths[u]], dtype=torch.int64, device=DEV)
        at = pool_rows(self.table, u, r, self.P)
        x = self.rows.view(-1, 512)[at]
        x = x.double() if self.row_scale is None else e4m3_rows(x, self.row_scale.view(-1)[at])
        return torch.cat((x, self.raw[self.U - u, :self.n_raw[u]].double()))

    def check(self, skip=None, units=None):
        for u in range(self.U) if units is None else units:
            x = self.values(u, (skip or {}).get(u, ()))
            check_attn(self.out[u], self.lse[u], *attn_reference(self.q[u], x, SCALE))


def some_lists(lengths, P, k, seed, order="ascending"):
    rng, lists = random.Random(seed), []
    for n in lengths:
        x = rng.sample(range(pages_of(n, P)), min(k, pages_of(n, P)))
        lists.append(sorted(x) if order == "ascending" else sorted(x, reverse=True) if order == "descending" else x)
    return lists


LENGTHS = [0, 1, 8, 47, 48, 49, 100, 257, 513, 1000]


@pytest.mark.parametrize("P", [8, 16, 32, 64, 128, 512, 4096])
@pytest.mark.parametrize("H,fp8,order", [(64, False, "ascending"), (64, False, "descending"), (128, False, "any"),
                                         (64, True, "any")])
def test_attention(cuda_lib, P, H, fp8, order):
    a = Attention(LENGTHS, some_lists(LENGTHS, P, 7, P, order), P, H, fp8, seed=P, top_k=9, pad=2)
    a(cuda_lib)
    status(cuda_lib)
    a.check()


@pytest.mark.parametrize("H,fp8", [(64, False), (128, False), (64, True), (128, True)])
def test_attention_of_a_batch(cuda_lib, H, fp8):
    rng = random.Random(5)
    lengths = [rng.choice((0, 1, rng.randint(0, 3000))) for _ in range(200)]
    a = Attention(lengths, some_lists(lengths, 64, 16, 6), 64, H, fp8)
    a(cuda_lib)
    status(cuda_lib)
    a.check(units=range(0, 200, 11))


def test_attention_equals_that_over_the_same_rows(cuda_lib):
    """All blocks in order are all rows: the dense call's bits."""
    lengths = [1000, 64, 1, 0, 500]
    a = Attention(lengths, [list(range(pages_of(n, 16))) for n in lengths], 16)
    a(cuda_lib)
    out, lse = torch.empty_like(a.out), torch.empty_like(a.lse)
    n = cuda_lib.ds4a_workspace_bytes(cuda_lib.DS4A_OP_PAGED_ATTN_DECODE, 5, 1, a.table.shape[1] * 16, 0)
    cuda_lib.ds4a_paged_attn_decode(a.q, a.rows, a.table, a.n_rows, a.raw, a.raw_n, SCALE, out, lse,
                                    torch.empty(n, dtype=torch.uint8, device=DEV), ring=a.ring)
    whole = [u for u, n in enumerate(lengths) if n % 16 == 0]    # (a ragged end makes other tiles)
    assert torch.equal(out[whole], a.out[whole]) and torch.equal(lse[whole], a.lse[whole])
    a.check()


def test_attention_of_a_block_listed_twice_and_of_one_long_list(cuda_lib):
    a = Attention([300, 5000], [[2, 2, 0], list(range(300))[::-1]], 16, top_k=313)
    a.lists[1] = [b for b in a.lists[1]]
    a(cuda_lib)
    status(cuda_lib)
    a.check()


def test_attention_of_nothing(cuda_lib):
    a = Attention([100, 0, 70], [[], [], []], 16, n_raw=[0, 0, 5], top_k=4)
    a(cuda_lib)
    status(cuda_lib)
    assert (a.out[:2] == 0).all() and torch.isneginf(a.lse[:2]).all()
    a.check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad", ["negative", "behind", "far", "page"])
def test_attention_of_blocks_that_are_not_there(cuda_lib, bad, fp8):
    a = Attention([500, 200], [[0, 3, 9, 31], [12, 1]], 16, fp8=fp8)
    if bad == "page":
        a.table[0, 3] = a.n_pages
    else:
        a.idx[0, 1] = {"negative": -3, "behind": 32, "far": 2 ** 31 - 1}[bad]
    a(cuda_lib)
    status(cuda_lib, BOUNDS)
    a.check(skip={0: (3,)})
    a.idx[0, 1] = 3
    a.table[0, 3] = a.table[0, 3] if bad != "page" else 0
    for count in (-1, 5):                            # a count out of range is clamped
        a.count[1] = count
        a.lists[1] = [] if count < 0 else [12, 1]
        if count > 0:
            a.idx[1, 2:] = ints([0, 5])
            a.lists[1] = [12, 1, 0, 5]
        a(cuda_lib)
        status(cuda_lib, BOUNDS)
        a.check(units=[1])


def test_attention_with_infinite_logits_and_nan_rows(cuda_lib):
    """Rows that are not listed may hold anything; a NaN row that is makes its heads NaN."""
    a = Attention([640, 640], [[0, 5, 7], [1, 2]], 64)
    at = int(a.table[0, 3])
    a.rows[at] = float("nan")
    a.rows[int(a.table[1, 2]), 5, 9] = float("nan")
    a(cuda_lib)
    a.check(units=[0])
    assert a.out[1].isnan().all() and a.lse[1].isnan().all()


def test_attention_captured_and_on_two_streams(cuda_lib):
    lengths = [3000, 100, 2000, 0, 700]
    a = Attention(lengths, some_lists(lengths, 32, 12, 9), 32, top_k=12)
    b = Attention([4000] * 40, some_lists([4000] * 40, 64, 20, 8), 64, seed=3)
    a(cuda_lib), b(cuda_lib)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a(cuda_lib)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for x in (a, b):
        x.out.zero_(), x.lse.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s):
            graph.replay()
        b(cuda_lib, stream=t)
    torch.cuda.synchronize()
    first = a.out.clone()
    a.check(), b.check(units=[0, 13, 39])
    lists = some_lists(lengths, 32, 5, 21)            # other lists through the same graph
    a.lists = lists
    a.idx.fill_(-1)
    for u, x in enumerate(lists):
        a.idx[u, :len(x)] = ints(x) if x else a.idx[u, :0]
    a.count.copy_(ints([len(x) for x in lists]))
    graph.replay()
    torch.cuda.synchronize()
    a.check()
    assert not torch.equal(first, a.out)


def test_rejects_other_tensors(cuda_lib):
    a = Attention([100, 64], [[0], [1, 2]], 16)
    a(cuda_lib)
    good = dict(q=a.q, rows=a.rows, table=a.table, n_rows=a.n_rows, block_idx=a.idx, block_count=a.count, raw=a.raw,
                n_raw=a.raw_n, scale=SCALE, out=a.out, lse=a.lse, ws=a.ws, ring=a.ring)
    for change in (dict(block_idx=None), dict(block_count=None), dict(block_idx=a.idx.long()), dict(block_count=a.count[:1]),
                   dict(q=a.q.float()), dict(rows=a.rows.half()), dict(out=a.out.float()), dict(ws=a.ws.cpu())):
        with pytest.raises(ValueError):
            cuda_lib.ds4a_paged_attn_blocks(**dict(good, **change))
    with pytest.raises(cuda_lib.Ds4aError):
        cuda_lib.ds4a_paged_attn_blocks(**dict(good, ws=None))
    k, s = KeyStore([100, 64], 16), Scores([7, 4], 8)
    good = dict(ik=k.ik, table=k.table, n_rows=k.n_rows, block_keys=k.block_keys, n_blocks=k.n_blocks)
    for change in (dict(ik=k.ik.half()), dict(table=k.table[:1]), dict(block_keys=k.block_keys[:-1]),
                   dict(block_keys=k.block_keys.float()), dict(n_blocks=k.n_blocks[:1]), dict(cu_row=k.n_rows),
                   dict(first_row=k.n_rows[:1]), dict(n_rows=k.n_rows.long())):
        with pytest.raises(ValueError):
            cuda_lib.ds4a_paged_block_keys(**dict(good, **change))
    good = dict(iq=s.iq, w=s.w, block_keys=s.keys, table=s.table, n_blocks=s.n_blocks, scores=s.scores)
    for change in (dict(iq=s.iq[:1]), dict(w=s.w.half()), dict(block_keys=s.keys[:, :64]), dict(table=s.table.long()),
                   dict(n_blocks=s.n_blocks[:1]), dict(scores=s.scores[:, 0])):
        with pytest.raises(ValueError):
            cuda_lib.ds4a_paged_block_score(**dict(good, **change))
    with pytest.raises(cuda_lib.Ds4aError):
        cuda_lib.ds4a_paged_block_score(**dict(good, n_first=-1))
    assert math.isfinite(float(a.lse.sum()))
