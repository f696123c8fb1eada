"""A NaN in a row or a query of the contiguous attention calls reaches the results it
belongs to, whether its unit is computed whole or in pieces that are joined."""
import pytest
import torch

from paged_util import DEV, gen, ints

pytestmark = pytest.mark.gpu
SCALE = 512 ** -0.5
MANY = 400                              # units: most of them whole; 1 and 3 are cut over the CTAs


class Calls:
    def __init__(self, lib, kind, U, H, n_rows=600, top_k=500):
        g = gen(U + H)
        self.lib, self.kind, self.U, self.H, self.top_k = lib, kind, U, H, top_k
        self.q = torch.randn(U, H, 512, generator=g, device=DEV).to(torch.bfloat16)
        shared = kind.startswith("prefill")
        self.rows = torch.randn(1 if shared else U, n_rows, 512, generator=g, device=DEV).to(torch.bfloat16)
        self.raw = torch.randn(1 if shared else U, 128, 512, generator=g, device=DEV).to(torch.float16)
        self.idx = torch.arange(top_k, dtype=torch.int32, device=DEV).repeat(U, 1) + 7
        self.n = ints([n_rows if kind == "dense" else top_k] * U)
        self.n_raw = ints([128] * U)
        self.q_pos = ints([127] * U)
        self.codes, self.row_scale = None, None
        if kind.endswith("fp8"):
            self.codes = (self.rows.float() * 100).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            self.row_scale = torch.full(self.codes.shape[:2], 2.0 ** -7, device=DEV)
        op = dict(dense=lib.DS4A_OP_DENSE_ATTN_DECODE, sparse=lib.DS4A_OP_SPARSE_ATTN_DECODE,
                  prefill=lib.DS4A_OP_SPARSE_ATTN_PREFILL)[kind.split("_")[0]]
        sizes = (1, U, n_rows, top_k) if shared else (U, 1, n_rows, 0 if kind == "dense" else top_k)
        n = lib.ds4a_workspace_bytes(op | (lib.DS4A_OP_FLAG_128_HEADS if H == 128 else 0), *sizes)
        self.ws = torch.full((max(n, 1),), 0x7F, dtype=torch.uint8, device=DEV)      # whatever it held before: NaN
        self.out, self.lse = torch.empty(U, H, 512, device=DEV), torch.empty(U, H, device=DEV)

    def __call__(self):
        lib, tail = self.lib, (SCALE, self.out, self.lse, self.ws)
        if self.kind == "dense":
            lib.ds4a_dense_attn_decode_heads(self.H, self.q, self.rows, self.n, self.raw, self.n_raw, *tail)
        elif self.kind == "sparse":
            lib.ds4a_sparse_attn_decode_heads(self.H, self.q, self.rows, self.idx, self.n, self.raw, self.n_raw, *tail)
        elif self.kind == "sparse_fp8":
            lib.ds4a_sparse_attn_decode_fp8(self.q, self.codes, self.row_scale, self.idx, self.n, self.raw, self.n_raw, *tail)
        elif self.kind == "prefill":
            lib.ds4a_sparse_attn_prefill_heads(self.H, self.q, self.q_pos, self.rows[0], self.idx, self.n, self.raw[0], 0, *tail)
        else:
            lib.ds4a_sparse_attn_prefill_fp8(self.q, self.q_pos, self.codes[0], self.row_scale[0], self.idx, self.n,
                                             self.raw[0], 0, *tail)
        assert lib.ds4a_get_device_status() == (0, 0)
        return torch.isnan(self.out), torch.isnan(self.lse)


@pytest.mark.parametrize("U", [1, 3, MANY])
@pytest.mark.parametrize("kind,H", [("dense", 64), ("dense", 128), ("sparse", 64), ("sparse", 128), ("sparse_fp8", 64),
                                    ("prefill", 64), ("prefill", 128), ("prefill_fp8", 64)])
def test_nan_stays(cuda_lib, kind, H, U):
    c = Calls(cuda_lib, kind, U, H)
    clean = [x.clone() for x in (c() and (c.out, c.lse))]
    assert torch.isfinite(clean[0]).all() and torch.isfinite(clean[1]).all()
    # one head's query, in the first and the last unit
    keep = c.q.clone()
    for u in {0, U - 1}:
        c.q[u, 9, 100] = float("nan")
    out, lse = c()
    want = torch.zeros(U, H, dtype=torch.bool, device=DEV)
    want[0, 9] = want[U - 1, 9] = True
    assert torch.equal(out.all(-1), want) and torch.equal(out.any(-1), want) and torch.equal(lse, want)
    assert torch.equal(c.out[~want], clean[0][~want]) and torch.equal(c.lse[~want], clean[1][~want])
    c.q.copy_(keep)
    # a row of the first unit (a chunk: of every query that lists it)
    if kind.endswith("fp8"):
        c.codes[0, 11, 7] = 0x7F
    else:
        c.rows[0, 11, 7] = float("nan")
    if kind.startswith("prefill") and U > 1:
        c.idx[1:] += 20                         # the first query alone lists row 11
    out, lse = c()
    assert out[0].all() and lse[0].all()
    assert not out[1:].any() and not lse[1:].any()
    if not kind.startswith("prefill"):
        assert torch.equal(c.out[1:], clean[0][1:]) and torch.equal(c.lse[1:], clean[1][1:])
