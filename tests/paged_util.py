"""Plain 64-bit references of the paged-cache operators and seeded paged inputs
(test helpers; torch and Python only, nothing of the library)."""
import math

import torch

DEV = "cuda"
WINDOW = 128


def gen(seed, device=DEV):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def ints(v, device=DEV):
    return torch.tensor(v, dtype=torch.int32, device=device)


def pages_of(n, P):
    return -(-n // P)


def make_table(lengths, P, max_pages, spare=2, seed=0, pad=0, device=DEV):
    """table [U, max_pages] (rows `max_pages + pad` apart) over a pool of just enough
    pages in random order; entries behind a unit's last page are -1.  Returns
    (table, number of pages, pages nobody holds)."""
    g = gen(seed, "cpu")
    need = [pages_of(n, P) for n in lengths]
    n_pages = sum(need) + spare
    perm = torch.randperm(n_pages, generator=g).tolist()
    full = torch.full((len(lengths), max_pages + pad), -1, dtype=torch.int32)
    at = 0
    for u, k in enumerate(need):
        full[u, :k] = torch.tensor(perm[at:at + k], dtype=torch.int32)
        at += k
    return full.to(device)[:, :max_pages], n_pages, perm[at:]


def pool_rows(table, u, rows, P):
    """Pool rows of unit u's rows (int64 tensor)."""
    r = rows.long()
    return table[u].long()[r // P] * P + r % P


# ------------------------------------------------------------------------------------------ plan
def plan_reference(past, add, ratio, P, free, head, table, ring, T_cap, R_cap):
    """The step's arrays by a walk over the sequences; `table` is a list of lists."""
    out = dict(n_rows=[], n_raw=[], cu_tok=[0], cu_row=[0], tok_pos=[], raw_slot=[], row_pos=[], row_slot=[])
    table = [list(t) for t in table]
    for b, (p, a) in enumerate(zip(past, add)):
        end = p + a
        old, new = p // ratio, end // ratio
        for i in range(pages_of(old, P), pages_of(new, P)):
            table[b][i] = free[head]
            head += 1
        for pos in range(p, end):
            out["tok_pos"].append(pos)
            out["raw_slot"].append((b if ring is None else ring[b]) * WINDOW + pos % WINDOW if pos >= end - WINDOW else -1)
        for j in range(old, new):
            out["row_pos"].append((j + 1) * ratio - 1)
            out["row_slot"].append(table[b][j // P] * P + j % P)
        out["n_rows"].append(new)
        out["n_raw"].append(min(end, WINDOW))
        out["cu_tok"].append(out["cu_tok"][-1] + a)
        out["cu_row"].append(out["cu_row"][-1] + new - old)
    for k, cap in (("tok_pos", T_cap), ("raw_slot", T_cap), ("row_pos", R_cap), ("row_slot", R_cap)):
        out[k] += [-1] * (cap - len(out[k]))
    return out, table, head


# ------------------------------------------------------------------------------- norm and rotation
def norm_rope_reference(x, weight, pos, inv_freq, eps, style):
    """x [T, heads, D] -> float64, and per element the size of the pair it was turned from."""
    x = x.double()
    D, n_rot = x.shape[-1], 2 * inv_freq.numel()
    y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + eps)
    if weight is not None:
        y = y * weight.double()
    size = y.abs()
    angle = pos.double()[:, None, None] * inv_freq
    c, s = torch.cos(angle), torch.sin(angle)
    i = torch.arange(n_rot // 2, device=x.device)
    a = D - n_rot + (2 * i if style == 0 else i)
    b = a + (1 if style == 0 else n_rot // 2)
    ya, yb = y[..., a], y[..., b]
    out = y.clone()
    out[..., a], out[..., b] = ya * c - yb * s, ya * s + yb * c
    both = ya.abs() + yb.abs()
    size[..., a], size[..., b] = both, both
    return out, size


# --------------------------------------------------------------------------------------- attention
def e4m3_rows(codes, scale):
    return codes.view(torch.float8_e4m3fn).double() * scale.double()[..., None]


def attn_reference(q, x, scale):
    """q [H, 512], x [n, 512] float64 -> out, lse, and sum_j a_j |x_j| and the largest sum_d |q_d x_d| scale."""
    H = q.shape[0]
    if x.shape[0] == 0:
        z = torch.zeros(H, x.shape[1], dtype=torch.float64, device=q.device)
        return z, torch.full((H,), -math.inf, dtype=torch.float64, device=q.device), z, 0.0
    q = q.double()
    z = q @ x.T * scale
    a = torch.softmax(z, -1)
    terms = float((q.abs() @ x.abs().T).max()) * abs(scale)
    return a @ x, torch.logsumexp(z, -1), a @ x.abs(), terms


def check_attn(out, lse, ref, ref_lse, absum, terms):
    """Bounds from the arithmetic (all relative to sum_j a_j |x_j|, per element):
    p rounded to bf16 (2^-8) before it multiplies a row; a logit is a sum of 512
    exact products in fp32, off by at most 512 * 2^-24 * sum_d |q_d x_d| scale = e,
    so a weight is off by a factor within e^(+-2e); 2^x and the fp32 sums add less
    than 2^-16.  The result is rounded once to bf16: 2^-8 of itself."""
    e = 512 * 2.0 ** -24 * terms
    rel = 2.0 ** -8 + math.expm1(2 * e) + 2.0 ** -16
    tol = rel * absum + 2.0 ** -8 * (ref.abs() + rel * absum) + 1e-30
    d = (out.double() - ref).abs()
    assert torch.isfinite(out.float()).all()
    assert (d <= tol).all(), f"out off by {float((d / tol).max()):.3f} of its bound"
    if lse is not None:
        fin = torch.isfinite(ref_lse)
        assert torch.equal(torch.isneginf(lse), torch.isneginf(ref_lse))
        t = e + 2.0 ** -16 + 2.0 ** -22 * ref_lse[fin].abs()
        assert ((lse.double()[fin] - ref_lse[fin]).abs() <= t).all()
