"""PagedDecodeStep: several decode steps of a growing, ragged, padded batch, each
stage against plain references on what the stage before it stored."""
import pytest
import torch

from paged_util import (DEV, WINDOW, attn_reference, check_attn, e4m3_rows, gen, ints, norm_rope_reference, plan_reference,
                        pool_rows)

pytestmark = pytest.mark.gpu
SCALE = 512 ** -0.5
EPS = 1e-6
FP32 = 2.0 ** -19                       # fp32 error of a rotated value, of its pair's size


class Program:
    """What a serving program keeps between steps."""

    def __init__(self, U, P, max_pages, n_pages, fp8, seed=0):
        g = self.g = gen(seed)
        self.U, self.P, self.fp8 = U, P, fp8
        n_ring = U + 2
        perm = torch.randperm(n_pages, generator=gen(seed, "cpu")).to(torch.int32)
        self.x = dict(
            table=torch.full((U, max_pages), -1, dtype=torch.int32, device=DEV), free_pages=perm.to(DEV),
            free_head=ints([0]), ring=torch.randperm(n_ring, generator=g, device=DEV)[:U].to(torch.int32),
            raw=torch.full((n_ring, WINDOW, 512), float("nan"), dtype=torch.float16, device=DEV),
            ik=torch.full((n_pages, P, 128), float("nan"), dtype=torch.bfloat16, device=DEV),
            inv_freq=10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64, device=DEV) / 64),
            past=ints([0] * U), add=ints([0] * U))
        for k, n in (("q_norm", 512), ("kv_norm", 512), ("iq_norm", 128), ("ik_norm", 128)):
            self.x[k] = 1 + 0.1 * torch.randn(n, generator=g, device=DEV)
        if fp8:
            self.x["rows"] = torch.full((n_pages, P, 512), 0x7F, dtype=torch.uint8, device=DEV)
            self.x["row_scale"] = torch.ones(n_pages, P, device=DEV)
        else:
            self.x["rows"] = torch.full((n_pages, P, 512), float("nan"), dtype=torch.bfloat16, device=DEV)

    def inputs(self, H):
        r = lambda *shape: torch.randn(*shape, generator=self.g, device=DEV)      # noqa: E731
        self.x.update(q=r(self.U, H, 512).to(torch.bfloat16), kv=r(self.U, 512).to(torch.bfloat16),
                      iq=r(self.U, 64, 128).to(torch.bfloat16), w=torch.rand(self.U, 64, generator=self.g, device=DEV),
                      pooled=r(self.U, 512), pooled_ik=r(self.U, 128))

    def stored(self, u, n):
        at = pool_rows(self.x["table"], u, torch.arange(n, device=DEV), self.P)
        if self.fp8:
            return e4m3_rows(self.x["rows"].view(-1, 512)[at], self.x["row_scale"].view(-1)[at])
        return self.x["rows"].view(-1, 512)[at].double()


def near(got, x, weight, pos, inv_freq, half, floor=0.0):
    ref, size = norm_rope_reference(x[:, None], weight, pos, inv_freq, EPS, 0)
    err = FP32 * size[:, 0]
    assert ((got.double() - ref[:, 0]).abs() <= err + half * (ref[:, 0].abs() + err) + floor).all()


@pytest.mark.parametrize("top_k,ratio,P,H,fp8", [(16, 4, 8, 64, False), (0, 4, 16, 128, False), (40, 2, 8, 64, True),
                                                 (0, 1, 64, 64, True)])
def test_steps(cuda_lib, top_k, ratio, P, H, fp8):
    import deepseek_v4_sparse_indexer_gb300 as pkg
    U, live, max_pages = 6, 4, 64
    p = Program(U, P, max_pages, 300, fp8)
    x = p.x
    step = pkg.PagedDecodeStep(U, max_pages, P, top_k=top_k, ratio=ratio, n_head=H, fp8=fp8)
    past, table, head = [0, 3, 0, 1, 0, 0], x["table"].tolist(), 0
    # a prompt's rows, stored by the same calls: 200 tokens for sequence 2, one for 0
    chunk, prompt = [1, 0, 200, 0, 0, 0], {}
    T = sum(chunk)
    names = ("n_rows", "n_raw", "cu_tok", "cu_row", "tok_pos", "raw_slot", "row_pos", "row_slot")
    for k, n in zip(names, (U, U, U + 1, U + 1, T, T, T, T)):
        prompt[k] = torch.empty(n, dtype=torch.int32, device=DEV)
    past[1] = past[3] = 0                        # (no row of theirs is stored yet)
    x["past"].copy_(ints(past)), x["add"].copy_(ints(chunk))
    pkg.ds4a_paged_plan(x["past"], x["add"], ratio, P, x["free_pages"], x["free_head"], x["table"], *[prompt[k] for k in names],
                        x["free_head"], ring=x["ring"])
    kv = torch.randn(T, 512, generator=p.g, device=DEV).to(torch.bfloat16)
    pkg.ds4a_qk_norm_rope(None, kv, prompt["tok_pos"], x["inv_freq"], EPS, None, x["kv_norm"], None, x["raw"].view(-1, 512),
                          k_slot=prompt["raw_slot"])
    rows = torch.randn(T, 512, generator=p.g, device=DEV)
    pkg.ds4a_qk_norm_rope(None, rows, prompt["row_pos"], x["inv_freq"], EPS, None, x["kv_norm"], None, x["rows"].view(-1, 512),
                          k_slot=prompt["row_slot"], k_scale=x["row_scale"].view(-1) if fp8 else None)
    keys = torch.randn(T, 128, generator=p.g, device=DEV)
    pkg.ds4a_qk_norm_rope(None, keys, prompt["row_pos"], x["inv_freq"], EPS, None, x["ik_norm"], None, x["ik"].view(-1, 128),
                          k_slot=prompt["row_slot"])
    want, table, head = plan_reference(past, chunk, ratio, P, x["free_pages"].tolist(), head, table, x["ring"].tolist(), T, T)
    for k in names:
        assert prompt[k].tolist() == want[k], k
    past = [a + b for a, b in zip(past, chunk)]
    add = [1] * live + [0] * (U - live)
    graph = None
    for n in range(2 * max(ratio, 4) + 3):
        p.inputs(H)
        if graph is None:
            bufs = {k: x[k].clone() for k in ("q", "kv", "iq", "w", "pooled", "pooled_ik")}
        for k in bufs:
            bufs[k].copy_(x[k])
        x.update(bufs)
        x["past"].copy_(ints(past)), x["add"].copy_(ints(add))
        before = step.q.clone()
        if n == 0:
            step(x, SCALE)
        elif graph is None:                      # the second step is captured, and replayed from then on
            state = {k: x[k].clone() for k in ("table", "free_head", "raw", "rows", "ik")}
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step(x, SCALE)
            for k, v in state.items():           # (capturing runs nothing)
                assert torch.equal(x[k].view(torch.uint8), v.view(torch.uint8))
            graph.replay()
        else:
            graph.replay()
        assert cuda_lib.ds4a_get_device_status() == (0, 0)
        want, table, head = plan_reference(past, add, ratio, P, x["free_pages"].tolist(), head, table, x["ring"].tolist(), U, U)
        for k in names:
            assert getattr(step, k).tolist() == want[k], k
        assert x["table"].tolist() == table and x["free_head"].item() == head
        pos = step.tok_pos[:live]
        near(x["raw"].view(-1, 512)[step.raw_slot[:live].long()], x["kv"][:live], x["kv_norm"], pos, x["inv_freq"], 2.0 ** -11,
             2.0 ** -25)
        ref, size = norm_rope_reference(x["q"][:live], x["q_norm"], pos, x["inv_freq"], EPS, 0)
        err = FP32 * size
        assert ((step.q[:live].double() - ref).abs() <= err + 2.0 ** -8 * (ref.abs() + err)).all()
        assert torch.equal(step.q[live:], before[live:])
        new = want["cu_row"][-1]
        if new:
            at = step.row_slot[:new].long()
            if not fp8:
                near(x["rows"].view(-1, 512)[at], x["pooled"][:new], x["kv_norm"], step.row_pos[:new], x["inv_freq"], 2.0 ** -8)
            if top_k:
                near(x["ik"].view(-1, 128)[at], x["pooled_ik"][:new], x["ik_norm"], step.row_pos[:new], x["inv_freq"],
                     2.0 ** -8)
        for u in range(U):
            rows = torch.arange(want["n_rows"][u], device=DEV)
            if top_k:
                sc = step.scores[u, 0, :len(rows)]
                at = pool_rows(x["table"], u, rows, P)
                k = x["ik"].view(-1, 128)[at].double()
                q = step.iq[u].double()
                ref = ((k @ q.T).relu() * x["w"][u].double()).sum(-1)
                tol = 194 * 2.0 ** -24 * ((k.abs() @ q.abs().T) * x["w"][u].double()).sum(-1) + 1e-30
                assert ((sc.double() - ref).abs() <= tol).all()
                rows = torch.topk(sc, min(top_k, len(rows))).indices.sort().values
                assert step.idx[u, 0, :len(rows)].tolist() == rows.tolist() and int(step.count[u]) == len(rows)
            kv = torch.cat((p.stored(u, want["n_rows"][u])[rows.long()], x["raw"][int(x["ring"][u]), :want["n_raw"][u]].double()))
            check_attn(step.out[u], step.lse[u], *attn_reference(step.q[u], kv, SCALE))
        past = [a + b for a, b in zip(past, add)]
