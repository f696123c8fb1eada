"""Operators around a paged decode step: what each is measured on, in plain torch and through the library.

  norm    the residual's addition, the RMS norm of the sum, and its output in 16 bits and as
          E4M3 codes with scales                                       ds4a_add_rms_norm
  keys    mean indexer key of each page that new rows went to          ds4a_paged_block_keys
  score   indexer scores of one new token over the blocks' mean keys   ds4a_paged_block_score
  attn    attention of one new token over the rows of listed blocks
          and the raw window                                           ds4a_paged_attn_blocks
  mass    the weights that this attention gave each row, summed over
          heads and added to what the steps before gave it             ds4a_paged_attn_mass
  evict   the rows that got least leave the cache: those that stay go
          to pages of their own, the old pages to the free list        ds4a_paged_evict

A cache of one layer is a pool of pages of P rows; table[u, i] is the page that holds rows i*P .. i*P+P-1
of unit u, in no order; a block is the rows of one page.  Lengths are spread evenly over their range and
dealt to the units by the seed, so that every seed has the same work.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DIM, IDX_HEADS, IDX_DIM, WINDOW = 512, 64, 128, 128
EPS = 1e-6
FIRST, LAST = 1, 2                # blocks at a list's ends that are selected whatever they score
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "none": 0, "e4m3": 1}


# ----------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one new token's hidden state before a layer's projections: latency
        dict(name="norm_token_1", op="norm", T=1, D=4096, x="bf16", res="bf16", out="bf16", group=128, pow2=True),
        # a batch of prompts, the residual kept in fp32, codes with a scale for each 128 for 8-bit projections
        dict(name="norm_prompt_8192", op="norm", T=8192, D=4096, x="bf16", res="fp32", out="none", group=128, pow2=False),
        # a decode step of a batch: each sequence's newest page
        dict(name="keys_decode_256", op="keys", B=256, N=16384, add=1, P=64),
        # prompts that fill their caches
        dict(name="keys_prompt_32", op="keys", B=32, N=16384, add=16384, P=64),
        # a batch of 32 sequences of up to 256k tokens, 1,024 blocks each
        dict(name="score_32x65536", op="score", U=32, N=65536, P=64),
        # long contexts in small pages, up to 16,384 blocks each
        dict(name="score_64x262144", op="score", U=64, N=262144, P=16),
        # a few sequences, 1,024 rows in 16 blocks each: latency
        dict(name="attn_8x16x64", op="attn", U=8, N=16384, H=64, P=64, rows="bf16", k=16),
        # a batch, 2,048 rows in 32 blocks each, 128 heads
        dict(name="attn_256x32x64", op="attn", U=256, N=16384, H=128, P=64, rows="bf16", k=32),
        # the ratio-4 layers: the weights of the 512 rows that the indexer listed
        dict(name="mass_list_16x512", op="mass", U=16, N=16384, H=64, P=64, rows="bf16", kind="rows", k=512),
        # the ratio-128 layers of a big batch: every row
        dict(name="mass_all_256x8192", op="mass", U=256, N=8192, H=64, P=64, rows="bf16", kind="all", k=0),
        # a few sequences, half of them over their limit
        dict(name="evict_4x4096", op="evict", B=4, N=4096, keep=2048, P=64, rows="bf16", ik=True, planes=1),
        # a batch, half of it over the limit, 128 heads
        dict(name="evict_64x16384", op="evict", B=64, N=16384, keep=8192, P=64, rows="bf16", ik=True, planes=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm", "keys", "score", "attn", "attn", "mass", "mass", "evict", "evict"))
    P = rng.choice((8, 16, 32, 64, 128, 256))
    if op == "norm":
        D = rng.choice((512, 1536, 2048, 4096, 7168, 8 * rng.randint(1, 2048)))
        out = rng.choice(("bf16", "fp32", "none"))
        group = rng.choice((128, 64, 32, 0))
        return dict(op=op, T=_log(rng, 1, min(16384, 2 ** 25 // D)), D=D, x=rng.choice(("bf16", "fp16", "fp32")),
                    res=rng.choice(("bf16", "fp32", "none")), out=out, group=group, pow2=bool(rng.randint(0, 1)))
    if op == "keys":
        B = _log(rng, 1, 512)
        N = _log(rng, 64, min(65536, 2 ** 20 // B))
        return dict(op=op, B=B, N=N, add=rng.choice((1, _log(rng, 1, N), N)), P=P)
    if op == "score":
        U = _log(rng, 1, 256)
        return dict(op=op, U=U, N=_log(rng, 8 * P, min(2 ** 20, 2 ** 20 * P // U)), P=P)
    if op == "evict":
        B = _log(rng, 1, 96)
        keep = _log(rng, 64, min(8192, 2 ** 18 // B))
        return dict(op=op, B=B, N=rng.randint(keep + 1, 3 * keep), keep=keep, P=P, rows=rng.choice(("bf16", "e4m3")),
                    ik=bool(rng.randint(0, 1)), planes=rng.randint(1, 2))
    U, H = _log(rng, 1, 256), rng.choice((64, 128))
    rows = rng.choice(("bf16", "bf16", "e4m3"))
    if op == "attn":
        k = _log(rng, 1, max(1, min(256, 2 ** 18 // (U * P))))
        return dict(op=op, U=U, N=_log(rng, P, min(16384, 2 ** 21 // U)), H=H, P=P, rows=rows, k=k)
    kind = rng.choice(("all", "rows", "blocks"))
    N = _log(rng, 64, min(16384, 2 ** 26 // (U * H)))
    k = 0 if kind == "all" else _log(rng, 1, min(N, 1024)) if kind == "rows" else _log(rng, 1, max(1, min(N, 2048) // P))
    return dict(op=op, U=U, N=N, H=H, P=P, rows=rows, kind=kind, k=k)


def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi], both ends among them (one number: hi)."""
    return [hi - ((hi - lo) * i) // max(n - 1, 1) for i in range(n)]


def _pages(n, P):
    return (n + P - 1) // P


def _lengths(case):
    n = case.get("U", case.get("B"))
    if case["op"] == "evict":
        return _spread(case["keep"] // 2, case["N"], n)
    return _spread(0 if n > 4 else 1, case["N"], n)


def _new_rows(case):
    """New rows of each sequence, by length from the longest down."""
    return [min(n, case["add"]) if case["add"] == 1 or i % 2 == 0 else min(n, case["add"] // 3)
            for i, n in enumerate(_lengths(case))]


def _evict_sizes(case):
    """(limit, first rows kept, last rows kept)"""
    keep = case["keep"]
    return keep + keep // 8, min(4, keep // 4), keep // 8


# ---------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, d, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype) * (1.0 / math.sqrt(d))


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _table(g, lengths, cap, P, spare=3):
    """A random table for these lengths over a pool of just enough pages and `spare` more, and the pages in
    the order they were dealt (those that no unit holds last)."""
    need = [_pages(n, P) for n in lengths]
    n_pages = sum(need) + spare
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    cols = max(1, _pages(cap, P))
    needed = _ints(need)
    start = torch.cumsum(needed, 0) - needed
    i = torch.arange(cols, device=DEV)
    at = (start[:, None] + i[None, :]).clamp_(max=n_pages - 1)
    table = torch.where(i[None, :] < needed[:, None], perm[at], -1).to(torch.int32)
    return table.contiguous(), n_pages, perm


def _rows(g, kind, n_pages, P):
    """Normalised rows (rms 1), bf16 or E4M3 codes with a scale per row."""
    if kind == "e4m3":
        codes = (_normal(g, (n_pages, P, DIM), 1, torch.bfloat16) * 100).clamp_(-448, 448).to(torch.float8_e4m3fn)
        scale = torch.exp2(torch.randint(-8, -5, (n_pages, P), generator=g, device=DEV).float())
        return codes.view(torch.uint8), scale
    return _normal(g, (n_pages, P, DIM), 1, torch.bfloat16), None


def _list_of(g, most, n_of, k):
    """k of each unit's first n_of[u] numbers (all of them where it has fewer), ascending, then -1; their count."""
    j = torch.arange(most, device=DEV)
    sc = torch.rand(n_of.numel(), most, generator=g, device=DEV).masked_fill_(j[None, :] >= n_of[:, None], -1.0)
    top, at = torch.topk(sc, min(k, most), dim=1)
    at = torch.where(top >= 0, at, most).sort(dim=1).values
    idx = torch.full((n_of.numel(), k), -1, dtype=torch.int32, device=DEV)
    idx[:, :at.shape[1]] = torch.where(at < most, at, -1).to(torch.int32)
    return idx, (top >= 0).sum(1).to(torch.int32)


def prepare(case, seed):
    g, r = _gen(seed), random.Random(seed)
    s = dict(case)
    if case["op"] == "norm":
        T, D = case["T"], case["D"]
        s["hidden"] = _normal(g, (T, D), 1, torch.float32).mul_(3).to(TYPES[case["x"]])
        s["weight"] = 1 + 0.1 * _normal(g, (D,), 1, torch.float32)
        s["residual"] = s["res_out"] = s["out_rows"] = None
        if case["res"] != "none":
            s["residual"] = _normal(g, (T, D), 1, torch.float32).mul_(5).to(TYPES[case["res"]])
            s["res_out"] = torch.zeros_like(s["residual"])
        if case["out"] != "none":
            s["out_rows"] = torch.zeros(T, D, dtype=TYPES[case["out"]], device=DEV)
        groups = _pages(D, case["group"]) if case["group"] else 1
        s["codes"] = torch.zeros(T, D, dtype=torch.uint8, device=DEV)
        s["scales"] = torch.ones(T, groups, device=DEV)
        s["n_live"] = _ints([T - 3 if T > 16 else T])          # a padded batch
        return s
    P = case["P"]
    lengths = _lengths(case)
    if case["op"] == "keys":
        both = list(zip(lengths, _new_rows(case)))
        r.shuffle(both)
        lengths = [n for n, _ in both]
        s["n_rows"] = _ints(lengths)
        s["cu_row"] = torch.cat((s["n_rows"].new_zeros(1), torch.cumsum(_ints([a for _, a in both]), 0).to(torch.int32)))
        s["table"], n_pages, _ = _table(g, lengths, case["N"], P)
        s["ik"] = _normal(g, (n_pages, P, IDX_DIM), IDX_DIM, torch.bfloat16)
        # one key more than the store has, for what the plain form leaves out
        s["keys"] = torch.zeros(n_pages + 1, IDX_DIM, dtype=torch.bfloat16, device=DEV)
        s["n_blocks"] = torch.zeros(case["B"], dtype=torch.int32, device=DEV)
        return s
    r.shuffle(lengths)
    s["n_rows"] = _ints(lengths)
    if case["op"] == "score":
        U, NB = case["U"], _pages(case["N"], P)
        s["n_blocks"] = _ints([_pages(n, P) for n in lengths])
        s["table"], n_pages, unused = _table(g, lengths, case["N"], P)
        s["iq"] = _normal(g, (U, 1, IDX_HEADS, IDX_DIM), IDX_DIM, torch.bfloat16)
        s["w"] = torch.rand(U, 1, IDX_HEADS, generator=g, device=DEV)
        s["keys"] = _normal(g, (n_pages, IDX_DIM), IDX_DIM, torch.bfloat16)
        s["scores"] = torch.full((U, 1, NB), -math.inf, device=DEV)
        return s
    if case["op"] == "evict":
        B, keep, N, planes = case["B"], case["keep"], case["N"], case["planes"]
        limit = _evict_sizes(case)[0]
        held = sum(_pages(n, P) for n in lengths)
        s["table"], n_pages, perm = _table(g, lengths, N, P, spare=sum(n > limit for n in lengths) * _pages(keep, P) + 3)
        s["rows_pool"], s["rows_scale"] = _rows(g, case["rows"], n_pages, P)
        s["ik_pool"] = _normal(g, (n_pages, P, IDX_DIM), IDX_DIM, torch.bfloat16) if case["ik"] else None
        # most rows get little, a few much; a mass is a sum of weights over many steps
        s["mass"] = torch.rand(planes, B, s["table"].shape[1] * P, generator=g, device=DEV).pow_(4).mul_(100)
        s["free"], s["head"] = perm, _ints([held])
        s["gone"] = torch.randint(0, 100, (B,), generator=g, device=DEV).to(torch.int32)
        for k, like in (("mass_out", "mass"), ("table_out", "table"), ("free_out", "free"), ("head_out", "head"),
                        ("gone_out", "gone"), ("n_rows_out", "n_rows")):
            s[k] = torch.zeros_like(s[like])
        return s
    U, N, H, k = case["U"], case["N"], case["H"], case["k"]
    s["table"], n_pages, unused = _table(g, lengths, N, P)
    s["q"] = _normal(g, (U, H, DIM), 1, torch.bfloat16)
    s["rows_pool"], s["rows_scale"] = _rows(g, case["rows"], n_pages, P)
    s["scale"] = 1.0 / math.sqrt(DIM)
    s["idx"] = s["count"] = None
    if case["op"] == "attn":
        s["idx"], s["count"] = _list_of(g, s["table"].shape[1], (s["n_rows"] + P - 1) // P, k)
        n_ring = U + 2
        s["raw"] = _normal(g, (n_ring, WINDOW, DIM), 1, torch.float16)
        s["ring"] = torch.randperm(n_ring, generator=g, device=DEV)[:U].to(torch.int32)
        s["n_raw"] = _ints(_raw_lengths(U))
        s["out"] = torch.empty(U, H, DIM, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(U, H, device=DEV)
        return s
    if case["kind"] == "rows":
        s["idx"], s["count"] = _list_of(g, N, s["n_rows"], k)
    elif case["kind"] == "blocks":
        s["idx"], s["count"] = _list_of(g, s["table"].shape[1], (s["n_rows"] + P - 1) // P, k)
    # what the attention returns for logits of variance 1 over so many rows and the raw window
    n_att = s["n_rows"].float() if s["idx"] is None else s["count"].float() * (P if case["kind"] == "blocks" else 1)
    s["lse"] = (torch.log(n_att + WINDOW) + 0.5)[:, None] + 0.2 * _normal(g, (U, H), 1, torch.float32)
    s["mass"] = torch.rand(H // 64, U, s["table"].shape[1] * P, generator=g, device=DEV)
    return s


def _raw_lengths(U):
    n_raw = [WINDOW if i % 4 else (i * 37) % (WINDOW + 1) for i in range(U)]
    n_raw[0] = WINDOW
    return n_raw


# ------------------------------------------------------------------------------------ plain forms
def _plain_norm(s):
    T, D, group = s["T"], s["D"], s["group"] or s["D"]
    h = s["hidden"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    groups = s["scales"].shape[1]
    z = y.new_zeros(T, groups * group)
    z[:, :D] = y
    z = z.view(T, groups, group)
    amax = z.abs().amax(-1)
    if s["pow2"]:
        m, k = torch.frexp(amax)
        e = torch.where(m <= 0.875, k - 9, k - 8)
        scale = torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, 0).clamp(-126, 127))
        inv = 1.0 / scale
    else:
        scale = torch.where(amax > 0, amax / 448.0, 1.0)
        inv = torch.where(amax > 0, 448.0 / amax, 1.0)
    codes = (z * inv[..., None]).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(T, -1)[:, :D]
    live = torch.arange(T, device=DEV)[:, None] < s["n_live"]
    if s["residual"] is not None:
        s["res_out"].copy_(torch.where(live, h.to(s["res_out"].dtype), s["res_out"]))
    if s["out_rows"] is not None:
        s["out_rows"].copy_(torch.where(live, y.to(s["out_rows"].dtype), s["out_rows"]))
    s["codes"].copy_(torch.where(live, codes, s["codes"]))
    s["scales"].copy_(torch.where(live, scale, s["scales"]))


def _plain_keys(s):
    P, table, n = s["P"], s["table"].long(), s["n_rows"].long()
    new = s["cu_row"][1:].long() - s["cu_row"][:-1].long()
    begin, end = (n - new) // P, (n + P - 1) // P                       # blocks to do: begin .. end - 1
    cols = table.shape[1]
    i = torch.arange(min(cols, _pages(s["add"], P) + 1), device=DEV)
    block = begin[:, None] + i[None, :]
    todo = (block < end[:, None]) & (new[:, None] > 0)
    page = torch.gather(table, 1, block.clamp(max=cols - 1)).clamp(min=0)
    rows = s["ik"][page].float()                                        # [B, blocks, P, 128]
    there = torch.arange(P, device=DEV) < (n[:, None, None] - block[..., None] * P)
    mean = rows.masked_fill_(~there[..., None], 0.0).sum(2) / there.sum(2, keepdim=True).clamp(min=1)
    s["keys"][torch.where(todo, page, s["keys"].shape[0] - 1)] = mean.to(torch.bfloat16)
    s["n_blocks"].copy_(end)


def _plain_score(s):
    x = s["keys"][s["table"].long().clamp(min=0)].float()               # [U, blocks, 128]
    dots = torch.matmul(x, s["iq"][:, 0].float().transpose(1, 2))
    scores = torch.matmul(dots.clamp_(min=0), s["w"][:, 0, :, None])[..., 0]
    i, n = torch.arange(x.shape[1], device=DEV)[None, :], s["n_blocks"][:, None]
    scores = scores.masked_fill_((i < FIRST) | (i >= n - LAST), math.inf)
    s["scores"][:, 0].copy_(torch.where(i < n, scores, s["scores"][:, 0]))


def _plain_rows(s, kind):
    """The attended rows in fp32 [U, n, 512] (masked ones zero), which of them count, and their numbers."""
    table, P, U = s["table"], s["P"], s["table"].shape[0]
    if kind == "all":
        j = torch.arange(table.shape[1] * P, device=DEV)[None, :].expand(U, -1)
        there = j < s["n_rows"][:, None]
    elif kind == "rows":
        j = s["idx"].long().clamp(min=0)
        there = torch.arange(j.shape[1], device=DEV)[None, :] < s["count"][:, None]
    else:
        j = (s["idx"].long().clamp(min=0)[..., None] * P + torch.arange(P, device=DEV)).flatten(1)
        there = (torch.arange(j.shape[1], device=DEV)[None, :] < s["count"][:, None] * P) & (j < s["n_rows"][:, None])
    at = torch.gather(table, 1, j // P).long().clamp(min=0) * P + j % P
    x = s["rows_pool"].view(-1, DIM)[at]
    if s["rows_scale"] is not None:
        x = x.view(torch.float8_e4m3fn).float() * s["rows_scale"].view(-1)[at][..., None]
    return x.float().masked_fill_(~there[..., None], 0.0), there, j


def _plain_attn(s):
    x, there, _ = _plain_rows(s, "blocks")
    raw = s["raw"][s["ring"].long()].float()
    window = torch.arange(WINDOW, device=DEV)[None, :] < s["n_raw"][:, None]
    there = torch.cat((there, window), 1)
    x = torch.cat((x, raw.masked_fill_(~window[..., None], 0.0)), 1)
    logits = torch.matmul(s["q"].float(), x.transpose(1, 2)).mul_(s["scale"])
    logits.masked_fill_(~there[:, None, :], -math.inf)
    top = logits.amax(-1, keepdim=True).clamp(min=-3e38)
    p = logits.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    s["out"].copy_(torch.matmul(p, x) / torch.where(total > 0, total, 1.0))
    s["lse"].copy_(torch.where(total > 0, total.log() + top, -math.inf)[..., 0])


def _plain_mass(s):
    x, there, j = _plain_rows(s, s["kind"])
    p = torch.matmul(s["q"].float(), x.transpose(1, 2)).mul_(s["scale"]).sub_(s["lse"][..., None]).exp_()
    U, H, n = p.shape
    p = p.view(U, H // 64, 64, n).sum(2).masked_fill_(~there[:, None, :], 0.0).transpose(0, 1)   # [planes, U, n]
    s["mass"].scatter_add_(2, j[None].expand(H // 64, -1, -1), p)


def _plain_evict(s):
    P, keep, B = s["P"], s["keep"], s["B"]
    limit, first, recent = _evict_sizes(s)
    n, table = s["n_rows"].long(), s["table"].long()
    need = _pages(keep, P)
    s["n_rows_out"].copy_(torch.where(n > limit, keep, n))
    s["gone_out"].copy_(s["gone"] + torch.where(n > limit, n - keep, 0))
    out = (n > limit).nonzero()[:, 0]
    E = out.numel()
    n, held = n[out], (n[out] + P - 1) // P
    head = s["head"].long()
    head_out = head + E * need - held.sum()
    s["head_out"].copy_(head_out)
    if E == 0:
        return
    # rows that stay: the protected ends, then the greatest masses (of equal ones the lower row)
    mass = s["mass"][:, out]
    j = torch.arange(mass.shape[2], device=DEV)[None, :]
    rank = mass.sum(0).masked_fill_((j < first) | (j >= n[:, None] - recent), math.inf).masked_fill_(j >= n[:, None], -math.inf)
    src = rank.sort(dim=1, descending=True, stable=True).indices[:, :keep].sort(dim=1).values
    moved = torch.where(j < n[:, None], 0.0, s["mass_out"][:, out])
    moved[:, :, :keep] = torch.gather(mass, 2, src[None].expand(mass.shape[0], -1, -1))
    s["mass_out"][:, out] = moved
    # their new pages
    pages = s["free"].long()[head + torch.arange(E * need, device=DEV)].view(E, need)
    old = table[out]
    i = torch.arange(keep, device=DEV)
    at = torch.gather(old, 1, src // P) * P + src % P
    to = pages[:, i // P] * P + i % P
    for name in ("rows_pool", "rows_scale", "ik_pool"):
        if s[name] is not None:
            flat = s[name].view(-1, DIM if name == "rows_pool" else IDX_DIM) if s[name].dim() == 3 else s[name].view(-1)
            flat[to] = flat[at]
    s["table_out"][out[:, None], torch.arange(need, device=DEV)[None, :]] = pages.to(torch.int32)
    # the old pages, in front of the list's head
    i = torch.arange(old.shape[1], device=DEV)[None, :]
    s["free_out"][head_out + torch.arange(int(held.sum()), device=DEV)] = old[i < held[:, None]].to(torch.int32)


# --------------------------------------------------------------------------------------- one pass
def _answer(s):
    op = s["op"]
    if op == "norm":                         # the codes as the numbers that they are, next to their scales
        got = {"scales": s["scales"], "values": s["codes"].view(torch.float8_e4m3fn)}
        if s["res_out"] is not None:
            got["residual"] = s["res_out"]
        if s["out_rows"] is not None:
            got["out"] = s["out_rows"]
        return got
    if op == "keys":
        return {"keys": s["keys"][:-1], "n_blocks": s["n_blocks"]}
    if op == "score":
        return {"scores": s["scores"]}
    if op == "attn":
        return {"out": s["out"], "lse": s["lse"]}
    if op == "mass":
        return {"mass": s["mass"]}
    got = {k: s[k] for k in ("mass_out", "n_rows_out", "table_out", "free_out", "head_out", "gone_out", "rows_pool")}
    for k in ("rows_scale", "ik_pool"):
        if s[k] is not None:
            got[k] = s[k]
    return got


def run(s):
    op = s["op"]
    if not own:
        {"norm": _plain_norm, "keys": _plain_keys, "score": _plain_score, "attn": _plain_attn, "mass": _plain_mass,
         "evict": _plain_evict}[op](s)
        return _answer(s)
    import deepseek_v4_sparse_indexer_gb300 as pkg
    if op == "norm":
        pkg.ds4a_add_rms_norm(s["hidden"], s["weight"], EPS, out=s["out_rows"], residual=s["residual"], res_out=s["res_out"],
                              codes=s["codes"], scales=s["scales"], group=s["group"],
                              scale_style=pkg.DS4A_SCALE_POW2 if s["pow2"] else pkg.DS4A_SCALE_MAX, n_live=s["n_live"])
    elif op == "keys":
        pkg.ds4a_paged_block_keys(s["ik"], s["table"], s["n_rows"], s["keys"][:-1], s["n_blocks"], cu_row=s["cu_row"])
    elif op == "score":
        pkg.ds4a_paged_block_score(s["iq"], s["w"], s["keys"], s["table"], s["n_blocks"], s["scores"], n_first=FIRST,
                                   n_last=LAST)
    elif op == "attn":
        if "ws" not in s:                    # the program's workspace, kept
            kind = pkg.DS4A_OP_PAGED_ATTN_BLOCKS | (pkg.DS4A_OP_FLAG_128_HEADS if s["H"] == 128 else 0)
            n = pkg.ds4a_workspace_bytes(kind, s["U"], 1, s["k"] * s["P"], 0)
            s["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
        pkg.ds4a_paged_attn_blocks(s["q"], s["rows_pool"], s["table"], s["n_rows"], s["idx"], s["count"], s["raw"],
                                   s["n_raw"], s["scale"], s["out"], s["lse"], s["ws"], row_scale=s["rows_scale"],
                                   ring=s["ring"])
    elif op == "mass":
        pkg.ds4a_paged_attn_mass(s["q"], s["rows_pool"], s["table"], s["n_rows"], s["scale"], s["lse"], s["mass"],
                                 idx=s["idx"], count=s["count"], blocks=s["kind"] == "blocks", row_scale=s["rows_scale"])
    else:
        limit, first, recent = _evict_sizes(s)
        if "ws" not in s:
            n = pkg.ds4a_workspace_bytes(pkg.DS4A_OP_PAGED_EVICT, s["B"], 1, s["table"].shape[1] * s["P"], s["keep"])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        pkg.ds4a_paged_evict(s["mass"], s["n_rows"], s["table"], s["rows_pool"], s["free"], s["head"], s["keep"], limit,
                             s["mass_out"], s["n_rows_out"], s["table_out"], s["free_out"], s["head_out"], s["ws"],
                             first=first, recent=recent, row_scale=s["rows_scale"], ik=s["ik_pool"], gone=s["gone"],
                             gone_out=s["gone_out"])
    return _answer(s)


# ------------------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "norm":
        T, D = case["T"], case["D"]
        wide = BYTES[case["x"]] + 2 * BYTES[case["res"]] + BYTES[case["out"]] + 1
        groups = _pages(D, case["group"]) if case["group"] else 1
        return {"bytes": T * D * wide + 4 * T * groups + 4 * D, "flops": 7 * T * D}
    P, lengths = case["P"], _lengths(case)
    if op == "keys":
        rows = blocks = 0
        for n, a in zip(lengths, _new_rows(case)):
            if a:
                begin = (n - a) // P
                rows += n - begin * P
                blocks += _pages(n, P) - begin
        return {"bytes": rows * IDX_DIM * 2 + blocks * (IDX_DIM * 2 + 4) + 12 * case["B"], "flops": rows * IDX_DIM}
    if op == "score":
        blocks, U = sum(_pages(n, P) for n in lengths), case["U"]
        return {"bytes": blocks * (IDX_DIM * 2 + 8) + U * IDX_HEADS * (IDX_DIM * 2 + 4),
                "flops": blocks * IDX_HEADS * (2 * IDX_DIM + 3)}
    wide = DIM + 4 if case["rows"] == "e4m3" else DIM * 2
    if op == "evict":
        limit, keep = _evict_sizes(case)[0], case["keep"]
        over = [n for n in lengths if n > limit]
        b = len(over) * keep * 2 * (wide + (IDX_DIM * 2 if case["ik"] else 0))
        b += sum(4 * case["planes"] * (2 * n) + 4 * _pages(n, P) * 2 for n in over) + 16 * len(lengths)
        return {"bytes": b, "flops": sum(n * case["planes"] for n in over)}
    U, H = case["U"], case["H"]
    if op == "mass":
        n = [n if case["kind"] == "all" else min(n, case["k"] * (P if case["kind"] == "blocks" else 1)) for n in lengths]
        rows = sum(n)
        listed = 0 if case["kind"] == "all" else 4 * U * case["k"]
        return {"bytes": rows * (wide + 8 * H // 64) + U * H * (DIM * 2 + 4) + listed, "flops": rows * H * (2 * DIM + 3)}
    rows = sum(min(n, case["k"] * P) for n in lengths) + sum(_raw_lengths(U))
    raws = sum(_raw_lengths(U))
    return {"bytes": (rows - raws) * wide + raws * DIM * 2 + U * H * (DIM * 4 + 4) + 4 * U * case["k"],
            "flops": rows * H * (4 * DIM + 5)}


# -------------------------------------------------------------------- the definitions, in 64 bits
def _exact_norm(s):
    T, D, live = s["T"], s["D"], int(s["n_live"])
    h = s["hidden"][:live].double() + (s["residual"][:live].double() if s["residual"] is not None else 0.0)
    y = h / (h.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * s["weight"].double()
    amax = torch.stack([part.abs().amax(-1) for part in y.split(s["group"] or D, 1)], 1)
    scales = torch.ones(T, amax.shape[1], dtype=torch.float64, device=DEV)
    scales[:live] = torch.exp2(torch.ceil(torch.log2(amax / 448))) if s["pow2"] else amax / 448
    got = {"scales": scales, "values": None}             # the codes are held in 8 bits: their scales alone have a value
    for name, kept, v in (("residual", s["res_out"], h), ("out", s["out_rows"], y)):
        if kept is not None:
            got[name] = torch.zeros(T, D, dtype=torch.float64, device=DEV)
            got[name][:live] = v
    return got


def _exact_listed(s, u, kind):
    """The numbers of the rows that unit u attends to."""
    n, P = int(s["n_rows"][u]), s["P"]
    if kind == "all":
        return torch.arange(n, device=DEV)
    listed = s["idx"][u, :int(s["count"][u])].long()
    if kind == "rows":
        return listed
    r = (listed[:, None] * P + torch.arange(P, device=DEV)[None, :]).flatten()
    return r[r < n]


def _exact_rows(s, u, r):
    at = s["table"][u].long()[r // s["P"]] * s["P"] + r % s["P"]
    x = s["rows_pool"].view(-1, DIM)[at]
    if s["rows_scale"] is None:
        return x.double()
    return x.view(torch.float8_e4m3fn).to(torch.float64) * s["rows_scale"].view(-1)[at].double()[:, None]


def exact(case, seed):
    op = case["op"]
    if op == "evict":
        return None                          # rows and masses are copied, the rest are whole numbers
    s = prepare(case, seed)
    if op == "norm":
        return _exact_norm(s)
    P = s["P"]
    if op == "keys":
        keys = s["keys"][:-1].double()
        cu = s["cu_row"].tolist()
        table = s["table"].tolist()
        for b, n in enumerate(s["n_rows"].tolist()):
            if cu[b + 1] > cu[b]:
                begin = (n - (cu[b + 1] - cu[b])) // P
                pages = torch.tensor(table[b][begin:_pages(n, P)], device=DEV)
                rows = s["ik"][pages].double().view(-1, IDX_DIM)[:n - begin * P]
                whole = rows.shape[0] // P
                keys[pages[:whole]] = rows[:whole * P].view(whole, P, IDX_DIM).mean(1)
                if rows.shape[0] % P:
                    keys[pages[whole]] = rows[whole * P:].mean(0)
        return {"keys": keys, "n_blocks": None}
    if op == "score":
        scores = s["scores"].double()
        for u, n in enumerate(s["n_blocks"].tolist()):
            k = s["keys"][s["table"][u, :n].long()].double()
            scores[u, 0, :n] = ((k @ s["iq"][u, 0].double().T).relu() * s["w"][u].double()).sum(-1)
            scores[u, 0, :min(FIRST, n)] = math.inf
            scores[u, 0, max(n - LAST, 0):n] = math.inf
        return {"scores": scores}
    if op == "mass":
        mass, H = s["mass"].double(), case["H"]
        for u in range(case["U"]):
            r = _exact_listed(s, u, case["kind"])
            z = s["q"][u].double() @ _exact_rows(s, u, r).T * s["scale"]
            p = torch.exp(z - s["lse"][u].double()[:, None])
            mass[:, u, r] += p.view(H // 64, 64, r.numel()).sum(1)
        return {"mass": mass}
    out = torch.zeros(case["U"], case["H"], DIM, dtype=torch.float64, device=DEV)
    lse = torch.full((case["U"], case["H"]), -math.inf, dtype=torch.float64, device=DEV)
    n_raw, ring = s["n_raw"].tolist(), s["ring"].tolist()
    for u in range(case["U"]):
        x = torch.cat((_exact_rows(s, u, _exact_listed(s, u, "blocks")), s["raw"][ring[u], :n_raw[u]].double()))
        if x.shape[0]:
            z = s["q"][u].double() @ x.T * s["scale"]
            out[u], lse[u] = torch.softmax(z, -1) @ x, torch.logsumexp(z, -1)
    return {"out": out, "lse": lse}
