"""PagedDecodeStep with blocks, masses and eviction: captured steps of a growing,
ragged batch whose sequences are cut whenever they pass their limit, each stage
against plain references on what the stage before it stored."""
import pytest
import torch

from paged_util import (DEV, WINDOW, attn_reference, check_attn, e4m3_rows, gen, ints, make_table, pages_of, plan_reference,
                        pool_rows)

pytestmark = pytest.mark.gpu
SCALE = 512 ** -0.5


@pytest.mark.parametrize("blocks,top_k,H,fp8", [(4, 0, 64, False), (3, 0, 128, True), (0, 24, 64, False), (0, 0, 128, False)])
def test_steps(cuda_lib, blocks, top_k, H, fp8):
    import deepseek_v4_sparse_indexer_gb300 as pkg
    U, P, ratio, max_pages, evict = 5, 8, 2, 9, (40, 56, 2, 8)
    g = gen(H + blocks)
    past = [100, 113, 5, 0, 90]
    held = [p // ratio for p in past]
    gone = [0] * U
    table, _, _ = make_table(held, P, max_pages, seed=3)
    n_pages = 90
    taken = [int(table[u, i]) for u in range(U) for i in range(pages_of(held[u], P))]
    free = taken + [p for p in range(n_pages) if p not in taken]
    x = dict(table=table.contiguous(), free_pages=ints(free), free_head=ints([len(taken)]), past=ints(past), add=ints([0] * U),
             raw=torch.randn(U, WINDOW, 512, generator=g, device=DEV).to(torch.float16),
             ik=torch.full((n_pages, P, 128), float("nan"), dtype=torch.bfloat16, device=DEV),
             block_keys=torch.full((n_pages, 128), float("nan"), dtype=torch.bfloat16, device=DEV),
             inv_freq=10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64, device=DEV) / 64),
             mass=torch.zeros(H // 64, U, max_pages * P, device=DEV), gone=ints(gone))
    if fp8:
        x["rows"] = torch.full((n_pages, P, 512), 0x7F, dtype=torch.uint8, device=DEV)
        x["row_scale"] = torch.full((n_pages, P), 2.0 ** -7, device=DEV)
    else:
        x["rows"] = torch.full((n_pages, P, 512), float("nan"), dtype=torch.bfloat16, device=DEV)
    for u, n in enumerate(held):                 # what earlier steps stored
        at = pool_rows(x["table"], u, torch.arange(n, device=DEV), P)
        r = torch.randn(n, 512, generator=g, device=DEV)
        x["rows"].view(-1, 512)[at] = (r * 100).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else r.to(torch.bfloat16)
        x["ik"].view(-1, 128)[at] = torch.randn(n, 128, generator=g, device=DEV).to(torch.bfloat16)
    n_blocks = torch.empty(U, dtype=torch.int32, device=DEV)
    pkg.ds4a_paged_block_keys(x["ik"], x["table"], ints(held), x["block_keys"], n_blocks)
    for k, shape, t in (("q", (U, H, 512), torch.bfloat16), ("kv", (U, 512), torch.bfloat16),
                        ("iq", (U, 64, 128), torch.bfloat16), ("w", (U, 64), torch.float32),
                        ("pooled", (U, 512), torch.float32), ("pooled_ik", (U, 128), torch.float32)):
        x[k] = torch.empty(*shape, dtype=t, device=DEV)
    step = pkg.PagedDecodeStep(U, max_pages, P, top_k=top_k, ratio=ratio, n_head=H, fp8=fp8, pooled_by_sequence=True,
                               blocks=blocks, keep_blocks=(1, 1), mass=True, evict=evict)

    def value(u, rows):
        at = pool_rows(x["table"], u, rows, P)
        r = x["rows"].view(-1, 512)[at]
        return e4m3_rows(r, x["row_scale"].view(-1)[at]) if fp8 else r.double()

    def check_block_keys(lengths):
        for u, n in enumerate(lengths):
            for b in range(pages_of(n, P)):
                page = int(x["table"][u, b])
                k = x["ik"][page, :min(P, n - b * P)].double()
                err = 10 * 2.0 ** -24 * k.abs().mean(0)
                ref = k.mean(0)
                assert ((x["block_keys"][page].double() - ref).abs() <= err + 2.0 ** -8 * (ref.abs() + err)).all()

    graphs, evictions, head = None, 0, len(taken)
    for n in range(24):
        add = [1, 1, int(n % 3 == 0), int(n > 4), 1]
        for k in ("q", "kv", "iq", "pooled", "pooled_ik"):
            x[k].copy_(torch.randn(x[k].shape, generator=g, device=DEV))
        x["w"].copy_(torch.rand(U, 64, generator=g, device=DEV))
        x["past"].copy_(ints(past)), x["add"].copy_(ints(add))
        tables, before = x["table"].tolist(), x["mass"].clone()
        free = x["free_pages"].tolist()
        if n == 0:
            step(x, SCALE)
        else:
            if graphs is None:
                torch.cuda.synchronize()
                graphs = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
                with torch.cuda.graph(graphs[0]):
                    step(x, SCALE)
                with torch.cuda.graph(graphs[1]):
                    step.evict(x)
            graphs[0].replay()
        assert cuda_lib.ds4a_get_device_status() == (0, 0)
        virtual = [p - s * ratio for p, s in zip(past, gone)]
        want, tables, head = plan_reference(virtual, add, ratio, P, free, head, tables, None, U, U)
        assert step.n_rows.tolist() == want["n_rows"] and x["table"].tolist() == tables and x["free_head"].item() == head
        assert step.n_raw.tolist() == [min(p + a, WINDOW) for p, a in zip(past, add)]
        lengths = want["n_rows"]
        if blocks:
            check_block_keys(lengths)
        for u in range(U):
            if blocks:
                m = pages_of(lengths[u], P)
                sc = step.scores[u, 0, :m]
                k = x["block_keys"][x["table"][u, :m].long()].double()
                ref = ((k @ step.iq[u].double().T).relu() * x["w"][u].double()).sum(-1)
                tol = 194 * 2.0 ** -24 * ((k.abs() @ step.iq[u].double().abs().T) * x["w"][u].double()).sum(-1) + 1e-30
                inner = torch.arange(m, device=DEV)[1:-1]
                assert ((sc.double() - ref).abs() <= tol)[inner].all()
                chosen = sc.sort(descending=True, stable=True).indices[:blocks].sort().values
                assert step.idx[u, 0, :chosen.numel()].tolist() == chosen.tolist() and int(step.count[u]) == chosen.numel()
                rows = (chosen[:, None] * P + torch.arange(P, device=DEV)).flatten()
                rows = rows[rows < lengths[u]]
            elif top_k:
                rows = step.idx[u, 0, :int(step.count[u])].long()
                assert rows.numel() == min(top_k, lengths[u])
            else:
                rows = torch.arange(lengths[u], device=DEV)
            kv = torch.cat((value(u, rows), x["raw"][u, :min(past[u] + add[u], WINDOW)].double()))
            ref = attn_reference(step.q[u], kv, SCALE)
            check_attn(step.out[u], step.lse[u], *ref)
            # masses: of the rows attended to, of the units with a token
            want_mass = before[:, u].double()
            if add[u]:
                w = torch.exp(step.q[u].double() @ value(u, rows).T * SCALE - step.lse[u].double()[:, None])
                want_mass.index_add_(1, rows, w.view(H // 64, 64, rows.numel()).sum(1))
            assert ((x["mass"][:, u].double() - want_mass).abs() <= 2.0 ** -12 * want_mass.abs() + 1e-30).all()
        past = [p + a for p, a in zip(past, add)]
        # ---- eviction
        keep, limit, first, recent = evict
        kept = {}
        for u in range(U):
            if lengths[u] > limit:
                mass = x["mass"][:, u].sum(0).tolist()
                rank = sorted(range(first, lengths[u] - recent), key=lambda r: (-mass[r], r))[:keep - first - recent]
                kept[u] = sorted(list(range(first)) + rank + list(range(lengths[u] - recent, lengths[u])))
        old = {u: value(u, torch.arange(lengths[u], device=DEV)) for u in range(U)}
        old_keys = {u: x["ik"].view(-1, 128)[pool_rows(x["table"], u, torch.arange(lengths[u], device=DEV), P)] for u in range(U)}
        old_mass = x["mass"].clone()
        if graphs is None:
            step.evict(x)
        else:
            graphs[1].replay()
        assert cuda_lib.ds4a_get_device_status() == (0, 0)
        for u in range(U):
            at = torch.tensor(kept.get(u, list(range(lengths[u]))), dtype=torch.int64, device=DEV)
            assert torch.equal(value(u, torch.arange(at.numel(), device=DEV)), old[u][at])
            want_mass = old_mass[:, u].clone()
            if u in kept:
                gone[u] += lengths[u] - keep
                evictions += 1
                want_mass.zero_()
                want_mass[:, :keep] = old_mass[:, u, at]
            if blocks or top_k:
                now = x["ik"].view(-1, 128)[pool_rows(x["table"], u, torch.arange(at.numel(), device=DEV), P)]
                assert torch.equal(now, old_keys[u][at])
            assert torch.equal(x["mass"][:, u], want_mass)
        lengths = [keep if u in kept else m for u, m in enumerate(lengths)]
        assert x["gone"].tolist() == gone and step.n_rows.tolist() == lengths
        head = x["free_head"].item()
        # every page is in one table or in the list, once
        mine = [int(x["table"][u, i]) for u in range(U) for i in range(pages_of(lengths[u], P))]
        assert sorted(mine + x["free_pages"].tolist()[head:]) == list(range(n_pages))
        if blocks:
            check_block_keys(lengths)
    assert evictions >= 2
