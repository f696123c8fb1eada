"""The paged decode step's operators: what each is measured on, in plain torch and through the library.

  plan    block tables and slot maps from request lengths          ds4a_paged_plan
  rope    RMS norm of each query head and of the key row, tail
          rotation, the key stored at its slot, in one pass        ds4a_qk_norm_rope
  score   indexer scores of one new token over paged keys          ds4a_paged_indexer_score
  attn    attention of one new token over paged rows (all, or the
          indexer's list) and the raw window                       ds4a_paged_attn_decode

A cache of one layer is a pool of pages of P rows; table[u, i] is the page that holds rows i*P .. i*P+P-1
of unit u, in no order, and pages that no unit holds are filled with NaN.  Lengths are spread evenly over
their range and dealt to the units by the seed, so that every seed has the same work.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DIM, IDX_HEADS, IDX_DIM, WINDOW, N_ROT = 512, 64, 128, 128, 64
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}


# ----------------------------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step of a few sequences: latency
        dict(name="plan_decode_8", op="plan", B=8, past=65536, add=1, ratio=4, P=64),
        # many chunks of prompts at once, each up to the engine's 2,048 tokens
        dict(name="plan_prompts_256", op="plan", B=256, past=262144, add=2048, ratio=4, P=64),
        # one new token of one sequence: q of 64 heads, its row into the raw ring
        dict(name="rope_token_1", op="rope", T=1, H=64, D=512, q="bf16", k="bf16", store="ring", style=0),
        # a prompt chunk of 2,048 tokens: q of 64 heads, the last 128 rows into the ring
        dict(name="rope_chunk_2048", op="rope", T=2048, H=64, D=512, q="bf16", k="bf16", store="ring", style=0),
        # the indexer's queries of a chunk and the fp32 pooled keys into the paged key store
        dict(name="rope_indexer_2048", op="rope", T=2048, H=64, D=128, q="bf16", k="fp32", store="page", style=1),
        # pooled fp32 rows of many sequences into the paged FP8 row store
        dict(name="rope_rows_e4m3", op="rope", T=16384, H=0, D=512, q="bf16", k="fp32", store="page8", style=0),
        # the indexer over 8 sequences of up to 64k tokens
        dict(name="score_8x16384", op="score", U=8, N=16384, P=64),
        # a batch of 32 sequences of up to 256k tokens
        dict(name="score_32x65536", op="score", U=32, N=65536, P=64),
        # one short sequence, every row: latency
        dict(name="attn_all_1x1024", op="attn", U=1, N=1024, H=64, P=64, rows="bf16", k=0),
        # the ratio-128 layers of a big batch: every row, lengths of up to 1M tokens
        dict(name="attn_all_640x8192", op="attn", U=640, N=8192, H=64, P=64, rows="bf16", k=0),
        # the ratio-4 layers: the indexer's 1,024 rows of each unit, 128 heads
        dict(name="attn_list_128x16384", op="attn", U=128, N=16384, H=128, P=64, rows="bf16", k=1024),
        # FP8 rows in small pages, every row
        dict(name="attn_all_e4m3_48x4096", op="attn", U=48, N=4096, H=64, P=16, rows="e4m3", k=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("plan", "rope", "rope", "score", "score", "attn", "attn", "attn"))
    P = rng.choice((8, 16, 32, 64, 128, 256))
    if op == "plan":
        add = rng.choice((1, 1, _log(rng, 2, 2048)))
        B = _log(rng, 1, 256 if add > 1 else 4096)
        return dict(op=op, B=B, past=_log(rng, 1, 262144), add=add, ratio=rng.choice((4, 128)), P=P)
    if op == "rope":
        D = rng.choice((512, 512, 128))
        store = rng.choice(("ring", "page", "page8")) if D == 512 else "page"
        H = rng.choice((64, 128, rng.randint(1, 64), 0)) if D == 512 else 64
        T = _log(rng, 1, 2048 if H <= 64 else 1024) if H else _log(rng, 1, 16384)
        return dict(op=op, T=T, H=H, D=D, q=rng.choice(("bf16", "fp32")), k=rng.choice(("bf16", "fp32")),
                    store=store, style=rng.randint(0, 1))
    if op == "score":
        U = _log(rng, 1, 256)
        return dict(op=op, U=U, N=_log(rng, 64, min(262144, 2 ** 21 // U)), P=P)
    k = rng.choice((0, 0, _log(rng, 16, 1024)))
    U, H = _log(rng, 1, 512), rng.choice((64, 128))
    N = _log(rng, max(1, k), min(65536, 2 ** 28 // (U * H)))
    return dict(op=op, U=U, N=N, H=H, P=P, rows=rng.choice(("bf16", "bf16", "e4m3")), k=k)


def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi], both ends among them (one number: hi)."""
    return [hi - ((hi - lo) * i) // max(n - 1, 1) for i in range(n)]


def _pages(n, P):
    return (n + P - 1) // P


def _plan_sizes(case):
    B, ratio, P = case["B"], case["ratio"], case["P"]
    past = _spread(0, case["past"], B)
    add = [1] * B if case["add"] == 1 else _spread(0, case["add"], B)
    return past, add, ratio, P


# ---------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, d, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype) * (1.0 / math.sqrt(d))


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _inv_freq():
    return 10000.0 ** (-torch.arange(0, N_ROT, 2, dtype=torch.float64, device=DEV) / N_ROT)


def _table(g, lengths, cap, P, spare=3):
    """A random table for these lengths over a pool of just enough pages, and the pool's size."""
    need = [_pages(n, P) for n in lengths]
    n_pages = sum(need) + spare
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    cols = max(1, _pages(cap, P))
    needed = _ints(need)
    start = torch.cumsum(needed, 0) - needed
    i = torch.arange(cols, device=DEV)
    at = (start[:, None] + i[None, :]).clamp_(max=n_pages - 1)
    table = torch.where(i[None, :] < needed[:, None], perm[at], -1).to(torch.int32)
    return table.contiguous(), n_pages, perm[sum(need):].long()


def prepare(case, seed):
    g, r = _gen(seed), random.Random(seed)
    s = dict(case)
    if case["op"] == "plan":
        past, add, ratio, P = _plan_sizes(case)
        r.shuffle(past)
        r.shuffle(add)
        B = len(past)
        cols = max(1, _pages((max(past) + max(add)) // ratio, P))
        held = [_pages(p // ratio, P) for p in past]
        new = [_pages((p + a) // ratio, P) - h for p, a, h in zip(past, add, held)]
        pages = torch.randperm(sum(held) + sum(new) + 5, generator=g, device=DEV).to(torch.int32)
        have = _ints(held)
        start = torch.cumsum(have, 0) - have
        i = torch.arange(cols, device=DEV)
        at = (start[:, None] + i[None, :]).clamp_(max=pages.numel() - 1)
        s["table"] = torch.where(i[None, :] < have[:, None], pages[at], -1).to(torch.int32).contiguous()
        s["free"] = pages[sum(held):].contiguous()
        s["head"] = _ints([2])
        s["past"], s["add"] = _ints(past), _ints(add)
        s["ring"] = torch.randperm(B + 3, generator=g, device=DEV)[:B].to(torch.int32)
        # the program's fixed capacities: a few rows more than this step fills
        T, R = sum(add) + 7, sum(-(-a // ratio) for a in add) + 7
        for k, n in (("n_rows", B), ("n_raw", B), ("cu_tok", B + 1), ("cu_row", B + 1), ("tok_pos", T),
                     ("raw_slot", T), ("row_pos", R), ("row_slot", R), ("head_out", 1)):
            s[k] = torch.zeros(n, dtype=torch.int32, device=DEV)
        return s
    if case["op"] == "rope":
        T, H, D = case["T"], case["H"], case["D"]
        s["x"] = _normal(g, (T, H, D), 1, TYPES[case["q"]]) * 3 if H else None
        s["kx"] = _normal(g, (T, D), 1, TYPES[case["k"]]) * 2
        s["gq"] = 1 + 0.1 * _normal(g, (D,), 1, torch.float32)
        s["gk"] = 1 + 0.1 * _normal(g, (D,), 1, torch.float32)
        pos = torch.randint(0, 1 << 20, (T,), generator=g, device=DEV, dtype=torch.int32)
        if case["store"] == "ring":
            # one chunk of one sequence: consecutive positions, the last 128 rows kept
            pos = pos[:1] + torch.arange(T, device=DEV, dtype=torch.int32)
            slots = WINDOW * 4
            slot = torch.where(torch.arange(T, device=DEV) >= T - WINDOW, 2 * WINDOW + pos % WINDOW, -1)
        else:
            slots = T + T // 2 + 8
            slot = torch.randperm(slots, generator=g, device=DEV)[:T]
        if T > 16:   # a padded batch
            pos[T - 3:] = -1
            slot[T - 3:] = -1
        s["pos"], s["slot"] = pos.contiguous(), slot.to(torch.int32).contiguous()
        s["inv_freq"] = _inv_freq()
        s["q_out"] = torch.zeros(T, H, D, dtype=torch.bfloat16, device=DEV) if H else None
        # one row more than the store has, for what the plain form leaves out
        kind = {"ring": torch.float16, "page": torch.bfloat16, "page8": torch.uint8}[case["store"]]
        s["store_rows"] = torch.zeros(slots + 1, D, dtype=kind, device=DEV)
        s["store_scale"] = torch.ones(slots + 1, device=DEV) if case["store"] == "page8" else None
        return s
    U, N, P = case["U"], case["N"], case["P"]
    lengths = _spread(0 if U > 4 else 1, N, U)
    r.shuffle(lengths)
    s["n_rows"] = _ints(lengths)
    s["table"], n_pages, unused = _table(g, lengths, N, P)
    if case["op"] == "score":
        s["iq"] = _normal(g, (U, 1, IDX_HEADS, IDX_DIM), IDX_DIM, torch.bfloat16)
        s["w"] = torch.rand(U, 1, IDX_HEADS, generator=g, device=DEV)
        s["keys"] = _normal(g, (n_pages, P, IDX_DIM), IDX_DIM, torch.bfloat16)
        s["keys"][unused] = float("nan")
        s["scores"] = torch.full((U, 1, N), -math.inf, device=DEV)
        return s
    H, k = case["H"], case["k"]
    s["q"] = _normal(g, (U, H, DIM), 1, torch.bfloat16)           # normalised heads and rows: rms 1
    s["rows_scale"] = None
    if case["rows"] == "e4m3":
        s["rows"] = (_normal(g, (n_pages, P, DIM), 1, torch.bfloat16) * 100).clamp_(-448, 448).to(
            torch.float8_e4m3fn).view(torch.uint8)
        s["rows"][unused] = 0x7F
        s["rows_scale"] = torch.exp2(torch.randint(-8, -5, (n_pages, P), generator=g, device=DEV).float())
    else:
        s["rows"] = _normal(g, (n_pages, P, DIM), 1, torch.bfloat16)
        s["rows"][unused] = float("nan")
    n_ring = U + 2
    s["raw"] = _normal(g, (n_ring, WINDOW, DIM), 1, torch.float16)
    s["ring"] = torch.randperm(n_ring, generator=g, device=DEV)[:U].to(torch.int32)
    n_raw = [WINDOW if i % 4 else (i * 37) % (WINDOW + 1) for i in range(U)]
    n_raw[0] = WINDOW
    s["n_raw"] = _ints(n_raw)
    s["idx"] = s["count"] = None
    if k:
        # the k highest of random scores, ascending, then -1
        j = torch.arange(N, device=DEV)
        sc = torch.rand(U, N, generator=g, device=DEV).masked_fill_(j[None, :] >= s["n_rows"][:, None], -1.0)
        top, at = torch.topk(sc, k, dim=1)
        at = torch.where(top >= 0, at, N).sort(dim=1).values
        s["idx"] = torch.where(at < N, at, -1).to(torch.int32).contiguous()
        s["count"] = (top >= 0).sum(1).to(torch.int32)
    s["scale"] = 1.0 / math.sqrt(DIM)
    s["out"] = torch.empty(U, H, DIM, dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.empty(U, H, device=DEV)
    return s


# ------------------------------------------------------------------------------------ plain forms
def _plain_plan(s):
    past, add, ratio, P = s["past"].long(), s["add"].long(), s["ratio"], s["P"]
    table, B, cols = s["table"], s["past"].numel(), s["table"].shape[1]
    zero = past.new_zeros(1)
    old, new = past // ratio, (past + add) // ratio
    held, want = (old + P - 1) // P, (new + P - 1) // P
    cu_tok = torch.cat((zero, torch.cumsum(add, 0)))
    cu_row = torch.cat((zero, torch.cumsum(new - old, 0)))
    cu_page = torch.cat((zero, torch.cumsum(want - held, 0)))
    head = s["head"].long()
    # table entry (b, i) of a new page: the free list from the head on
    i = torch.arange(cols, device=DEV)[None, :]
    at = (head + cu_page[:B, None] + i - held[:, None]).clamp(0, s["free"].numel() - 1)
    fresh = (i >= held[:, None]) & (i < want[:, None])
    table.copy_(torch.where(fresh, s["free"][at], table))
    # tokens
    t = torch.arange(s["tok_pos"].numel(), device=DEV)
    b = torch.searchsorted(cu_tok, t, right=True).sub_(1).clamp_(max=B - 1)
    live = t < cu_tok[B]
    pos = past[b] + t - cu_tok[b]
    kept = live & (pos >= (past + add)[b] - WINDOW)
    s["tok_pos"].copy_(torch.where(live, pos, -1))
    s["raw_slot"].copy_(torch.where(kept, s["ring"].long()[b] * WINDOW + pos % WINDOW, -1))
    # rows
    t = torch.arange(s["row_pos"].numel(), device=DEV)
    b = torch.searchsorted(cu_row, t, right=True).sub_(1).clamp_(max=B - 1)
    live = t < cu_row[B]
    j = torch.where(live, old[b] + t - cu_row[b], 0)
    s["row_pos"].copy_(torch.where(live, j * ratio + ratio - 1, -1))
    s["row_slot"].copy_(torch.where(live, table[b, (j // P).clamp_(max=cols - 1)].long() * P + j % P, -1))
    s["n_rows"].copy_(new)
    s["n_raw"].copy_((past + add).clamp(max=WINDOW))
    s["cu_tok"].copy_(cu_tok)
    s["cu_row"].copy_(cu_row)
    s["head_out"].copy_(head + cu_page[B])


def _plain_norm_rope(x, weight, cos, sin, style):
    """x [T, heads, D] in any type, cos and sin [T, n_rot / 2] -> fp32."""
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
    tail = y[..., -N_ROT:]
    cos, sin = cos[:, None, :], sin[:, None, :]
    if style == 0:
        a, b = tail[..., 0::2], tail[..., 1::2]
        tail = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = tail[..., :N_ROT // 2], tail[..., N_ROT // 2:]
        tail = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((y[..., :-N_ROT], tail), -1)


def _plain_e4m3(y):
    """fp32 rows -> E4M3 codes and the smallest power-of-two scale with the row's maximum within 448."""
    amax = y.abs().amax(-1)
    m, k = torch.frexp(amax)
    e = torch.where(m <= 0.875, k - 9, k - 8)
    e = torch.where(amax > 0, e, 0).clamp(-126, 127)
    scale = torch.ldexp(torch.ones_like(amax), e)
    codes = (y / scale[..., None]).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), scale


def _plain_rope(s):
    angle = s["pos"].double()[:, None] * s["inv_freq"][None, :]
    cos, sin = angle.cos().float(), angle.sin().float()
    live = s["pos"] >= 0
    if s["x"] is not None:
        q = _plain_norm_rope(s["x"], s["gq"], cos, sin, s["style"])
        s["q_out"].copy_(torch.where(live[:, None, None], q, s["q_out"].float()))
    k = _plain_norm_rope(s["kx"][:, None], s["gk"], cos, sin, s["style"])[:, 0]
    rows = s["store_rows"]
    at = torch.where(live & (s["slot"] >= 0), s["slot"].long(), rows.shape[0] - 1)
    if s["store_scale"] is not None:
        codes, scale = _plain_e4m3(k)
        rows[at] = codes
        s["store_scale"][at] = scale
    else:
        rows[at] = k.to(rows.dtype)


def _plain_gather(pages, table, n_rows):
    """[U, columns * P, width] of the paged rows (in their own type) and which of them exist."""
    U, cols, P = table.shape[0], table.shape[1], pages.shape[1]
    x = pages[table.long().clamp(min=0)].view(U, cols * P, *pages.shape[2:])
    return x, torch.arange(cols * P, device=DEV)[None, :] < n_rows[:, None]


def _plain_score(s):
    x, there = _plain_gather(s["keys"], s["table"], s["n_rows"])
    dots = torch.matmul(x.float(), s["iq"][:, 0].float().transpose(1, 2))          # [U, rows, heads]
    scores = torch.matmul(dots.clamp_(min=0), s["w"][:, 0, :, None])[..., 0]
    N = s["N"]
    s["scores"][:, 0].copy_(torch.where(there[:, :N], scores[:, :N], s["scores"][:, 0]))


def _plain_attn(s):
    rows, table, P = s["rows"], s["table"], s["P"]
    U = table.shape[0]
    if s["idx"] is None:
        x, there = _plain_gather(rows, table, s["n_rows"])
        scale = None if s["rows_scale"] is None else _plain_gather(s["rows_scale"], table, s["n_rows"])[0]
    else:
        j = s["idx"].long().clamp(min=0)
        at = torch.gather(table, 1, j // P).long().clamp(min=0) * P + j % P
        x = rows.view(-1, DIM)[at]
        scale = None if s["rows_scale"] is None else s["rows_scale"].view(-1)[at]
        there = torch.arange(j.shape[1], device=DEV)[None, :] < s["count"][:, None]
    x = x.view(torch.float8_e4m3fn).float() * scale[..., None] if scale is not None else x.float()
    raw = s["raw"][s["ring"].long()].float()
    there = torch.cat((there, torch.arange(WINDOW, device=DEV)[None, :] < s["n_raw"][:, None]), 1)
    x = torch.cat((x, raw), 1).masked_fill_(~there[..., None], 0.0)                # [U, rows, 512]
    logits = torch.matmul(s["q"].float(), x.transpose(1, 2)).mul_(s["scale"])
    logits.masked_fill_(~there[:, None, :], -math.inf)
    top = logits.amax(-1, keepdim=True).clamp(min=-3e38)
    p = logits.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, x) / torch.where(total > 0, total, 1.0)
    s["out"].copy_(out)
    s["lse"].copy_(torch.where(total > 0, total.log() + top, -math.inf)[..., 0])


# --------------------------------------------------------------------------------------- one pass
def _answer(s):
    if s["op"] == "plan":
        return {k: s[k] for k in ("table", "n_rows", "n_raw", "cu_tok", "cu_row", "tok_pos", "raw_slot",
                                  "row_pos", "row_slot", "head_out")}
    if s["op"] == "rope":
        rows = s["store_rows"][:-1]
        if s["store_scale"] is not None:     # the values that the codes stand for
            rows = (rows.view(torch.float8_e4m3fn).float() * s["store_scale"][:-1, None]).to(torch.bfloat16)
        got = {"rows": rows} if s["x"] is None else {"q": s["q_out"], "rows": rows}
        return got if s["store_scale"] is None else dict(got, scale=s["store_scale"][:-1])
    if s["op"] == "score":
        return {"scores": s["scores"]}
    return {"out": s["out"], "lse": s["lse"]}


def run(s):
    if not own:
        {"plan": _plain_plan, "rope": _plain_rope, "score": _plain_score, "attn": _plain_attn}[s["op"]](s)
        return _answer(s)
    import deepseek_v4_sparse_indexer_gb300 as pkg
    if s["op"] == "plan":
        pkg.ds4a_paged_plan(s["past"], s["add"], s["ratio"], s["P"], s["free"], s["head"], s["table"], s["n_rows"],
                            s["n_raw"], s["cu_tok"], s["cu_row"], s["tok_pos"], s["raw_slot"], s["row_pos"],
                            s["row_slot"], s["head_out"], ring=s["ring"])
    elif s["op"] == "rope":
        scale = s["store_scale"]
        pkg.ds4a_qk_norm_rope(s["x"], s["kx"], s["pos"], s["inv_freq"], EPS, s["gq"], s["gk"], s["q_out"],
                              s["store_rows"][:-1], k_slot=s["slot"], k_scale=None if scale is None else scale[:-1],
                              style=s["style"])
    elif s["op"] == "score":
        pkg.ds4a_paged_indexer_score(s["iq"], s["w"], s["keys"], s["table"], s["n_rows"], s["scores"])
    else:
        if "ws" not in s:                    # the program's workspace, kept
            op = pkg.DS4A_OP_PAGED_ATTN_DECODE | (pkg.DS4A_OP_FLAG_128_HEADS if s["H"] == 128 else 0)
            n = pkg.ds4a_workspace_bytes(op, s["U"], 1, s["table"].shape[1] * s["P"], s["k"])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        pkg.ds4a_paged_attn_decode(s["q"], s["rows"], s["table"], s["n_rows"], s["raw"], s["n_raw"], s["scale"],
                                   s["out"], s["lse"], s["ws"], idx=s["idx"], count=s["count"],
                                   row_scale=s["rows_scale"], ring=s["ring"])
    return _answer(s)


# ------------------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "plan":
        past, add, ratio, P = _plan_sizes(case)
        B = len(past)
        T, R = sum(add) + 7, sum(-(-a // ratio) for a in add) + 7
        pages = sum(add) // (ratio * P)
        return {"bytes": 4 * (3 * B + 2 * B + 2 * (B + 1) + 2 * T + 2 * R + 2 * pages), "flops": 4 * (T + R)}
    if case["op"] == "rope":
        T, H, D = case["T"], case["H"], case["D"]
        kept = min(T, WINDOW) if case["store"] == "ring" else T
        wide = {"ring": 2, "page": 2, "page8": 1}[case["store"]]
        b = T * H * D * (BYTES[case["q"]] + 2) + kept * D * (BYTES[case["k"]] + wide)
        return {"bytes": b + 8 * T, "flops": 5 * D * (T * H + kept) + 4 * N_ROT * T * (H + 1)}
    rows = sum(_spread(0 if case["U"] > 4 else 1, case["N"], case["U"]))
    U = case["U"]
    if case["op"] == "score":
        return {"bytes": rows * (IDX_DIM * 2 + 4) + U * IDX_HEADS * (IDX_DIM * 2 + 4),
                "flops": rows * IDX_HEADS * (2 * IDX_DIM + 3)}
    if case["k"]:
        rows = sum(min(case["k"], n) for n in _spread(0 if U > 4 else 1, case["N"], U))
    n_raw = WINDOW + sum(WINDOW if i % 4 else (i * 37) % (WINDOW + 1) for i in range(1, U))
    b = rows * (DIM + 4 if case["rows"] == "e4m3" else DIM * 2) + n_raw * DIM * 2 + U * case["H"] * (DIM * 4 + 4)
    return {"bytes": b + (rows * 4 if case["k"] else 0), "flops": (rows + n_raw) * case["H"] * (4 * DIM + 5)}


# -------------------------------------------------------------------- the definitions, in 64 bits
def _exact_norm_rope(x, weight, pos, inv_freq, style):
    x = x.double()
    D = x.shape[-1]
    y = x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * weight.double()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos.double()[:, None] * inv_freq)
    first = torch.arange(N_ROT // 2, device=DEV) * (2 if style == 0 else 1) + D - N_ROT
    second = first + (1 if style == 0 else N_ROT // 2)
    z = torch.complex(y[..., first], y[..., second]) * (turn[:, None] if y.dim() == 3 else turn)
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    if case["op"] == "plan":
        return None                          # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "rope":
        live = s["pos"] >= 0
        got = {}
        if s["x"] is not None:
            q = _exact_norm_rope(s["x"], s["gq"], s["pos"], s["inv_freq"], s["style"])
            got["q"] = q * live[:, None, None]
        k = _exact_norm_rope(s["kx"], s["gk"], s["pos"], s["inv_freq"], s["style"])
        keep = s["slot"] >= 0
        if s["store_scale"] is None:
            rows = torch.zeros(s["store_rows"].shape[0] - 1, s["D"], dtype=torch.float64, device=DEV)
            rows[s["slot"][keep].long()] = k[keep]
            got["rows"] = rows
        else:                                # the codes are held in 8 bits: their scales alone have a value
            got["rows"] = None
            scale = torch.ones(s["store_rows"].shape[0] - 1, dtype=torch.float64, device=DEV)
            scale[s["slot"][keep].long()] = torch.exp2(torch.ceil(torch.log2(k[keep].abs().amax(-1) / 448)))
            got["scale"] = scale
        return got
    P, table = s["P"], s["table"].long()
    if case["op"] == "score":
        scores = s["scores"].double()
        keys = s["keys"].view(-1, IDX_DIM)
        for u, n in enumerate(s["n_rows"].tolist()):
            r = torch.arange(n, device=DEV)
            k = keys[table[u, r // P] * P + r % P].double()
            scores[u, 0, :n] = ((k @ s["iq"][u, 0].double().T).relu() * s["w"][u].double()).sum(-1)
        return {"scores": scores}
    rows = s["rows"].view(-1, DIM)
    out, lse = [], []
    n_rows, n_raw, ring = s["n_rows"].tolist(), s["n_raw"].tolist(), s["ring"].tolist()
    for u in range(case["U"]):
        r = torch.arange(n_rows[u], device=DEV) if s["idx"] is None else s["idx"][u, :int(s["count"][u])].long()
        at = table[u, r // P] * P + r % P
        if s["rows_scale"] is None:
            x = rows[at].double()
        else:
            x = rows[at].view(torch.float8_e4m3fn).to(torch.float64) * s["rows_scale"].view(-1)[at].double()[:, None]
        x = torch.cat((x, s["raw"][ring[u], :n_raw[u]].double()))
        z = s["q"][u].double() @ x.T * s["scale"]
        if not x.shape[0]:
            out.append(torch.zeros(case["H"], DIM, dtype=torch.float64, device=DEV))
            lse.append(torch.full((case["H"],), -math.inf, dtype=torch.float64, device=DEV))
            continue
        out.append(torch.softmax(z, -1) @ x)
        lse.append(torch.logsumexp(z, -1))
    return {"out": torch.stack(out), "lse": torch.stack(lse)}
