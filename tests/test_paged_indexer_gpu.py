"""ds4a_paged_indexer_score: the scores of ds4a_indexer_score over the same keys laid
out contiguously, bit for bit, and of the formula in 64 bits within the fp32
bound; entries that no row has left as they were."""
import random

import pytest
import torch

from paged_util import DEV, gen, ints, make_table, pages_of, pool_rows

pytestmark = pytest.mark.gpu


class Keys:
    def __init__(self, lengths, P, N_cap, seed=0, pad=0, max_pages=None):
        g, U = gen(seed), len(lengths)
        self.lengths, self.P, self.N_cap, self.U = lengths, P, N_cap, U
        self.table, self.n_pages, _ = make_table(lengths, P, max_pages or max(1, pages_of(max(lengths), P)), seed=seed, pad=pad)
        keys = torch.full((self.n_pages * P, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
        for u, n in enumerate(lengths):
            at = pool_rows(self.table, u, torch.arange(n, device=DEV), P)
            keys[at] = torch.randn(n, 128, generator=g, device=DEV).to(torch.bfloat16)
        self.ik = keys.view(self.n_pages, P, 128)
        self.iq = torch.randn(U, 1, 64, 128, generator=g, device=DEV).to(torch.bfloat16)
        self.w = torch.randn(U, 1, 64, generator=g, device=DEV)
        self.n_rows = ints(lengths)
        self.scores = torch.full((U, 1, N_cap), 7.0, device=DEV)

    def __call__(self, lib, stream=None):
        lib.ds4a_paged_indexer_score(self.iq, self.w, self.ik, self.table, self.n_rows, self.scores, stream=stream)

    def unit_keys(self, u):
        return self.ik.view(-1, 128)[pool_rows(self.table, u, torch.arange(self.lengths[u], device=DEV), self.P)]

    def check(self, lib, units=None, exact=True):
        units = list(range(self.U)) if units is None else units
        for u in units:
            n = self.lengths[u]
            assert (self.scores[u, 0, n:] == 7).all()
            if n == 0:
                continue
            k = self.unit_keys(u)
            q, w = self.iq[u, 0].double(), self.w[u, 0].double()
            ref = ((k.double() @ q.T).relu() * w).sum(-1)
            # 128 products, 64 weighted heads and 2 roundings in fp32
            tol = 194 * 2.0 ** -24 * ((k.double().abs() @ q.abs().T) * w.abs()).sum(-1) + 1e-30
            assert ((self.scores[u, 0, :n].double() - ref).abs() <= tol).all()
            if exact:
                same = torch.empty(1, 1, n, device=DEV)
                lib.ds4a_indexer_score(self.iq[u:u + 1], self.w[u:u + 1], k[None].contiguous(), ints([n]), same)
                assert torch.equal(same[0, 0], self.scores[u, 0, :n])


EDGES = [0, 1, 7, 8, 9, 127, 128, 129, 255, 256, 300, 1000]


@pytest.mark.parametrize("P", [8, 16, 32, 64, 128, 256, 4096])
def test_lengths_and_pages(cuda_lib, P):
    k = Keys(EDGES, P, 1003, pad=2, seed=P)
    k(cuda_lib)
    assert cuda_lib.ds4a_get_device_status() == (0, 0)
    k.check(cuda_lib)


@pytest.mark.parametrize("P", [16, 64])
def test_many_ragged_units(cuda_lib, P):
    rng = random.Random(1)
    lengths = [rng.choice((0, 0, 1, rng.randint(0, 2000))) for _ in range(500)]
    lengths[77] = 20000
    k = Keys(lengths, P, 20000)
    k(cuda_lib)
    assert cuda_lib.ds4a_get_device_status() == (0, 0)
    k.check(cuda_lib, units=list(range(0, 500, 7)) + [77])


def test_one_long_unit(cuda_lib):
    k = Keys([65536 - 5], 64, 65536)
    k(cuda_lib)
    k.check(cuda_lib)


@pytest.mark.parametrize("U", [1, 300])
def test_no_row_at_all(cuda_lib, U):
    k = Keys([0] * U, 64, 100)
    k(cuda_lib)
    assert cuda_lib.ds4a_get_device_status() == (0, 0)
    assert (k.scores == 7).all()


@pytest.mark.parametrize("P", [8, 64, 256])
@pytest.mark.parametrize("bad", [-1, "end", 2 ** 31 - 1])
def test_pages_outside_the_pool(cuda_lib, P, bad):
    k = Keys([700, 40], P, 700)
    k.table[0, 1] = k.n_pages if bad == "end" else bad
    k(cuda_lib)
    assert cuda_lib.ds4a_get_device_status() == (cuda_lib.DS4A_EDEVICE, cuda_lib.DS4A_DEV_BOUNDS)
    assert torch.isneginf(k.scores[0, 0, P:2 * P]).all()
    rows = torch.tensor([r for r in range(700) if r // P != 1], device=DEV)
    q, w = k.iq[0, 0].double(), k.w[0, 0].double()
    kk = k.ik.view(-1, 128)[pool_rows(k.table, 0, rows, P)].double()
    tol = 194 * 2.0 ** -24 * ((kk.abs() @ q.abs().T) * w.abs()).sum(-1)
    assert ((k.scores[0, 0, rows].double() - ((kk @ q.T).relu() * w).sum(-1)).abs() <= tol).all()
    k.check(cuda_lib, units=[1])


@pytest.mark.parametrize("n,limit", [(-4, 0), (129, 100), (2 ** 31 - 1, 100)])
def test_lengths_out_of_range(cuda_lib, n, limit):
    k = Keys([100, 128], 64, 100)                # the scores hold 100 rows
    k.lengths[1] = 100
    k.n_rows[0], k.n_rows[1] = n, 100
    k.lengths[0] = limit
    k(cuda_lib)
    assert cuda_lib.ds4a_get_device_status() == (cuda_lib.DS4A_EDEVICE, cuda_lib.DS4A_DEV_BOUNDS)
    k.check(cuda_lib)


def test_captured_and_selected(cuda_lib):
    """A captured scan and selection replayed on other lengths: the selection of the
    contiguous scan."""
    k = Keys([900, 1024, 500], 64, 1024, max_pages=16)
    idx, count = torch.empty(3, 1, 64, dtype=torch.int32, device=DEV), torch.empty(3, 1, dtype=torch.int32, device=DEV)
    k(cuda_lib)
    cuda_lib.ds4a_topk_select(k.scores, k.n_rows, 64, idx, count, None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        k(cuda_lib)
        cuda_lib.ds4a_topk_select(k.scores, k.n_rows, 64, idx, count, None)
    for lengths in ([900, 1024, 500], [0, 63, 500], [1, 700, 64]):
        k.lengths = lengths
        k.n_rows.copy_(ints(lengths))
        k.scores.fill_(7.0)
        graph.replay()
        k.check(cuda_lib)
        for u, n in enumerate(lengths):
            want = torch.topk(k.scores[u, 0, :n], min(n, 64)).indices.sort().values
            assert int(count[u]) == min(n, 64) and idx[u, 0, :min(n, 64)].tolist() == want.tolist()


def test_two_streams(cuda_lib):
    a, b = Keys([30000] * 3, 64, 30000, seed=1), Keys([2000] * 50, 16, 2000, seed=2)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a(cuda_lib, stream=s)
        b(cuda_lib, stream=t)
    torch.cuda.synchronize()
    a.check(cuda_lib)
    b.check(cuda_lib, units=[0, 20, 49])


def test_rejects_other_tensors(cuda_lib):
    k = Keys([100, 64], 64, 128)
    good = dict(iq=k.iq, w=k.w, ik=k.ik, table=k.table, n_rows=k.n_rows, scores=k.scores)
    for change in (dict(iq=k.iq.float()), dict(iq=k.iq.cpu()), dict(iq=k.iq[:1]), dict(w=k.w.half()), dict(w=k.w[:, :, :32]),
                   dict(ik=k.ik.half()), dict(ik=k.ik[:, :, :64]), dict(table=k.table.long()), dict(table=k.table[:1]),
                   dict(n_rows=k.n_rows[:1]), dict(scores=k.scores.half()), dict(scores=k.scores[:, 0]),
                   dict(scores=k.scores[:, :, ::2])):
        with pytest.raises(ValueError):
            cuda_lib.ds4a_paged_indexer_score(**dict(good, **change))
    with pytest.raises(cuda_lib.Ds4aError):
        cuda_lib.ds4a_paged_indexer_score(**dict(good, ik=k.ik.view(-1, 4, 128)))
