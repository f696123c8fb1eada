"""Dense decode attention of units long enough to be cut over every CTA (more than
128 pieces of one unit to join), against softmax attention in 64 bits."""
import pytest
import torch

from paged_util import DEV, attn_reference, gen, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_rows", [8063, 8193, 16401])
def test_one_long_unit(cuda_lib, n_rows):
    g, cap = gen(n_rows), n_rows + 7
    rows = torch.randn(1, cap, 512, generator=g, device=DEV).to(torch.bfloat16)
    q = torch.randn(1, 64, 512, generator=g, device=DEV).to(torch.bfloat16)
    raw = torch.randn(1, 128, 512, generator=g, device=DEV).to(torch.float16)
    out, lse = torch.empty(1, 64, 512, device=DEV), torch.empty(1, 64, device=DEV)
    ws = torch.empty(cuda_lib.ds4a_workspace_bytes(cuda_lib.DS4A_OP_DENSE_ATTN_DECODE, 1, 1, cap, 0), dtype=torch.uint8,
                     device=DEV)
    cuda_lib.ds4a_dense_attn_decode(q, rows, ints([n_rows]), raw, ints([128]), 512 ** -0.5, out, lse, ws)
    x = torch.cat((rows[0, :n_rows].double(), raw[0].double()))
    ref, ref_lse, absum, _ = attn_reference(q[0], x, 512 ** -0.5)
    # weights rounded to bf16 (2^-8 of sum_j a_j |x_j|); the rest is fp32
    assert ((out[0].double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -10) * absum).all()
    assert ((lse[0].double() - ref_lse).abs() <= 1e-3).all()
