"""PagedDecodeStep's options over several steps of a growing batch whose sequences take
turns, with and without a new token in any order: every projection against the
formula in 64 bits, and the attention against plain attention over what was stored."""
import random

import pytest
import torch

from paged_util import DEV, WINDOW, attn_reference, check_attn, e4m3_rows, gen, ints, norm_rope_reference, pages_of, pool_rows

pytestmark = pytest.mark.gpu
SCALE = 512 ** -0.5
EPS = 1e-6
FP32 = 2.0 ** -19                       # fp32 error of a rotated value, of its pair's size
U, P, MAX_PAGES = 7, 8, 16


def near(got, x, weight, pos, inv_freq, style, half, floor=0.0):
    """got [n, D] is x [n, D] (or per head) normalised and turned, rounded once by at most `half` of itself."""
    x = x[:, None] if x.dim() == 2 else x
    ref, size = norm_rope_reference(x, weight, pos, inv_freq, EPS, style)
    err = FP32 * size
    d = (got.double().view_as(ref) - ref).abs()
    assert (d <= err + half * (ref.abs() + err) + floor).all()


class Run:
    def __init__(self, pkg, fp8=False, top_k=24, ratio=4, H=64, by_seq=False, seed=0, **options):
        g = self.g = gen(seed)
        self.fp8, self.top_k, self.ratio, self.H, self.by_seq = fp8, top_k, ratio, H, by_seq
        n_pages = U * MAX_PAGES
        r = self.normal
        self.x = x = dict(
            table=torch.full((U, MAX_PAGES), -1, dtype=torch.int32, device=DEV),
            free_pages=torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32), free_head=ints([0]),
            ring=torch.randperm(U + 1, generator=g, device=DEV)[:U].to(torch.int32), past=ints([0] * U), add=ints([0] * U),
            raw=torch.full((U + 1, WINDOW, 512), float("nan"), dtype=torch.float16, device=DEV),
            ik=torch.full((n_pages, P, 128), float("nan"), dtype=torch.bfloat16, device=DEV),
            inv_freq=10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64, device=DEV) / 64))
        x["rows"] = torch.full((n_pages, P, 512), 0x7F, dtype=torch.uint8, device=DEV) if fp8 else \
            torch.full((n_pages, P, 512), float("nan"), dtype=torch.bfloat16, device=DEV)
        if fp8:
            x["row_scale"] = torch.ones(n_pages, P, device=DEV)
        for k, n in (("q_norm", 512), ("kv_norm", 512), ("iq_norm", 128), ("ik_norm", 128)):
            x[k] = 1 + 0.3 * r(n)
        self.draw()
        self.step = pkg.PagedDecodeStep(U, MAX_PAGES, P, top_k=top_k, ratio=ratio, n_head=H, fp8=fp8, eps=EPS,
                                        **(dict(options, pooled_by_sequence=True) if by_seq else options))

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.g, device=DEV)

    def draw(self):
        r = self.normal
        self.x.update(q=(3 * r(U, self.H, 512)).to(torch.bfloat16), kv=(2 * r(U, 512)).to(torch.bfloat16),
                      iq=(3 * r(U, 64, 128)).to(torch.bfloat16), w=torch.rand(U, 64, generator=self.g, device=DEV),
                      pooled=2 * r(U, 512), pooled_ik=2 * r(U, 128))

    # what the options say; a test of an option overrides the one that it changes
    idx_style = style = 0
    pooled_norm = "kv_norm"

    def row_pos(self, j):
        return (j + 1) * self.ratio - 1

    def check_index_queries(self, live, pos):
        near(self.step.iq[live], self.x["iq"][live], self.x["iq_norm"], pos, self.x["inv_freq"], self.idx_style, 2.0 ** -8)

    def check(self, past, add):
        x, s, inv = self.x, self.step, self.x["inv_freq"]
        live = [u for u in range(U) if add[u]]
        pos = ints([past[u] for u in live])
        if live:
            near(s.q[live], x["q"][live], x["q_norm"], pos, inv, self.style, 2.0 ** -8)
            at = [int(x["ring"][u]) * WINDOW + past[u] % WINDOW for u in live]
            near(x["raw"].view(-1, 512)[at], x["kv"][live], x["kv_norm"], pos, inv, self.style, 2.0 ** -11, 2.0 ** -25)
            if self.top_k:
                self.check_index_queries(live, pos)
        new = [u for u in live if (past[u] + 1) % self.ratio == 0]
        if new:
            src = new if self.by_seq else list(range(len(new)))
            j = [past[u] // self.ratio for u in new]
            row_pos = ints([self.row_pos(i) for i in j])
            at = [int(pool_rows(x["table"], u, torch.tensor([i], device=DEV), P)[0]) for u, i in zip(new, j)]
            if self.fp8:
                scale = x["row_scale"].view(-1)[at].double()
                got = e4m3_rows(x["rows"].view(-1, 512)[at], scale)
                near(got, x["pooled"][src], x[self.pooled_norm], row_pos, inv, self.style, 2.0 ** -4,
                     2.0 ** -10 * scale[:, None, None])
            else:
                near(x["rows"].view(-1, 512)[at], x["pooled"][src], x[self.pooled_norm], row_pos, inv, self.style, 2.0 ** -8)
            if self.top_k:
                near(x["ik"].view(-1, 128)[at], x["pooled_ik"][src], x["ik_norm"], row_pos, inv, self.idx_style, 2.0 ** -8)
        assert s.n_rows.tolist() == [(p + a) // self.ratio for p, a in zip(past, add)]
        for u in live:
            n = (past[u] + 1) // self.ratio
            rows = torch.arange(n, device=DEV)
            if self.top_k:
                k = x["ik"].view(-1, 128)[pool_rows(x["table"], u, rows, P)].double()
                q, w = s.iq[u].double(), x["w"][u].double()
                tol = 194 * 2.0 ** -24 * ((k.abs() @ q.abs().T) * w).sum(-1) + 1e-30
                assert ((s.scores[u, 0, :n].double() - ((k @ q.T).relu() * w).sum(-1)).abs() <= tol).all()
                rows = torch.topk(s.scores[u, 0, :n], min(self.top_k, n)).indices.sort().values
                assert int(s.count[u]) == len(rows) and s.idx[u, 0, :len(rows)].tolist() == rows.tolist()
            at = pool_rows(x["table"], u, rows, P)
            kv = e4m3_rows(x["rows"].view(-1, 512)[at], x["row_scale"].view(-1)[at]) if self.fp8 else \
                x["rows"].view(-1, 512)[at].double()
            kv = torch.cat((kv, x["raw"][int(x["ring"][u]), :min(past[u] + 1, WINDOW)].double()))
            check_attn(s.out[u], s.lse[u], *attn_reference(s.q[u], kv, SCALE))

    def steps(self, lib, n, seed=1):
        rng, past, graph = random.Random(seed), [0] * U, None
        x, kept = self.x, {k: self.x[k] for k in ("q", "kv", "iq", "w", "pooled", "pooled_ik")}
        for i in range(n):
            add = [int(rng.random() < 0.7) for _ in range(U)]
            self.draw()
            for k, v in kept.items():
                v.copy_(x[k])
                x[k] = v
            x["past"].copy_(ints(past)), x["add"].copy_(ints(add))
            if i == 1:                       # captured at its second step, replayed from then on
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    self.step(x, SCALE)
            self.step(x, SCALE) if graph is None else graph.replay()
            assert lib.ds4a_get_device_status() == (0, 0)
            self.check(past, add)
            past = [p + a for p, a in zip(past, add)]
        assert x["free_head"].item() == sum(pages_of(p // self.ratio, P) for p in past)


@pytest.mark.parametrize("by_seq", [False, True])
@pytest.mark.parametrize("fp8,top_k,ratio,H", [(False, 24, 4, 64), (True, 24, 2, 64), (False, 0, 1, 128), (True, 0, 4, 64)])
def test_any_order(cuda_lib, fp8, top_k, ratio, H, by_seq):
    import deepseek_v4_sparse_indexer_gb300 as pkg
    Run(pkg, fp8, top_k, ratio, H, by_seq).steps(cuda_lib, 40)


def test_fed_by_the_compressor(cuda_lib):
    """The pooled rows straight from ds4a_compressor_pool, one captured program for plan, pooling and store."""
    import deepseek_v4_sparse_indexer_gb300 as pkg
    run = Run(pkg, by_seq=True)
    x, ratio = run.x, run.ratio
    frontier = {k: torch.zeros(U, ratio, w, device=DEV) for k, w in (("kv", 512), ("score", 512), ("ik", 128), ("ik_score", 128))}

    def go():
        pkg.ds4a_compressor_pool(frontier["kv"], frontier["score"], x["pooled"])
        pkg.ds4a_compressor_pool(frontier["ik"], frontier["ik_score"], x["pooled_ik"])
        run.step(x, SCALE)
    rng, past, graph = random.Random(4), [0] * U, None
    for i in range(14):
        add = [int(rng.random() < 0.8) for _ in range(U)]
        for u in range(U):
            if add[u]:
                for k, v in frontier.items():
                    v[u, past[u] % ratio] = run.normal(v.shape[2])
        x["past"].copy_(ints(past)), x["add"].copy_(ints(add))
        if i == 1:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                go()
        go() if graph is None else graph.replay()
        assert cuda_lib.ds4a_get_device_status() == (0, 0)
        pooled = (torch.softmax(frontier["score"].double(), 1) * frontier["kv"].double()).sum(1)
        assert ((x["pooled"].double() - pooled).abs() <= 2.0 ** -14 * frontier["kv"].abs().amax(1)).all()
        run.check(past, add)
        past = [p + a for p, a in zip(past, add)]


class First(Run):
    def row_pos(self, j):
        return j * self.ratio


@pytest.mark.parametrize("by_seq", [False, True])
@pytest.mark.parametrize("ratio", [1, 4])
def test_rows_turned_by_their_first_token(cuda_lib, ratio, by_seq):
    import deepseek_v4_sparse_indexer_gb300 as pkg
    First(pkg, ratio=ratio, by_seq=by_seq, row_position="first").steps(cuda_lib, 20)
    with pytest.raises(ValueError):
        pkg.PagedDecodeStep(U, MAX_PAGES, P, row_position="middle")


@pytest.mark.parametrize("style,idx_style", [(0, 1), (1, 0), (1, None)])
def test_pairs_of_the_heads_and_of_the_indexer(cuda_lib, style, idx_style):
    import deepseek_v4_sparse_indexer_gb300 as pkg
    run = Run(pkg, style=style, idx_style=idx_style)
    run.style, run.idx_style = style, style if idx_style is None else idx_style
    run.steps(cuda_lib, 12)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ones", [False, True])
def test_pooled_rows_with_a_norm_of_their_own(cuda_lib, fp8, ones):
    import deepseek_v4_sparse_indexer_gb300 as pkg
    run = Run(pkg, fp8=fp8)
    run.x["row_norm"] = None if ones else 1 + 0.3 * run.normal(512)      # None: all ones
    run.pooled_norm = "row_norm"
    run.steps(cuda_lib, 12)


class GivenQueries(Run):
    def check_index_queries(self, live, pos):
        self.step.iq = self.x["iq"]              # what the scores are checked with; the step has no buffer of its own


def test_indexer_queries_as_given(cuda_lib):
    import deepseek_v4_sparse_indexer_gb300 as pkg
    run = GivenQueries(pkg, rotate_iq=False)
    assert not hasattr(run.step, "iq")
    run.steps(cuda_lib, 12)
    run.x["iq"] = run.x["iq"].float()
    with pytest.raises(ValueError):
        run.step(run.x, SCALE)


def test_more_wanted_than_the_table_holds(cuda_lib):
    """top_k above max_pages * page_size: every row is selected."""
    import deepseek_v4_sparse_indexer_gb300 as pkg
    Run(pkg, top_k=512, ratio=1).steps(cuda_lib, 12)


def test_on_a_stream_of_its_own(cuda_lib):
    """Every part of the step runs on the given stream: the results of the default one."""
    import deepseek_v4_sparse_indexer_gb300 as pkg
    runs = [Run(pkg, by_seq=True, seed=3) for _ in range(2)]
    side = torch.cuda.Stream()
    past = [0] * U
    for i in range(9):
        add = [(u + i) % 3 > 0 for u in range(U)]
        for run in runs:
            run.draw()
            run.x["past"].copy_(ints(past)), run.x["add"].copy_(ints([int(a) for a in add]))
        torch.cuda.synchronize()
        runs[0].step(runs[0].x, SCALE)
        runs[1].step(runs[1].x, SCALE, stream=side)
        torch.cuda.synchronize()
        live = [u for u in range(U) if add[u]]
        assert torch.equal(runs[0].step.out[live], runs[1].step.out[live])
        assert torch.equal(runs[0].step.idx[live], runs[1].step.idx[live])
        past = [p + int(a) for p, a in zip(past, add)]
    assert cuda_lib.ds4a_get_device_status() == (0, 0)
