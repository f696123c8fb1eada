"""FP8 rows whose weights differ by many powers of two: a dominant first row in
front of a long tail of equal-mean rows that are light one by one and heavy together.

Bounds: paged_util.check_attn, whose weights are off by half a step of bf16 relative
to themselves, however small they are."""
import pytest
import torch

from paged_util import DEV, WINDOW, attn_reference, check_attn, gen, ints, pages_of

pytestmark = pytest.mark.gpu
SCALE = 512 ** -0.5


def batch_of_whole_units(H):
    """So many units of one length that every share of the batch is one unit: none is cut into pieces."""
    return torch.cuda.get_device_properties(0).multi_processor_count * 64 // H


@pytest.mark.parametrize("H,n,head_scale,tail_scale,gaps", [
    (64, 65537, 2.0 ** 0, 2.0 ** -8, (9.0, 16.0)),       # 12 nats: the tail is 29 % of the mass
    (128, 65537, 2.0 ** 0, 2.0 ** -8, (9.0, 16.0)),
    (64, 262145, 2.0 ** -4, 2.0 ** -7, (13.0, 17.0)),    # 14.9 nats: 8 %
    (64, 4097, 2.0 ** 20, 2.0 ** -40, (20.0, 40.0)),     # scales far apart: the tail counts in the sum alone
])
@pytest.mark.parametrize("n_raw", [0, WINDOW])
def test_long_light_tail(cuda_lib, H, n, head_scale, tail_scale, gaps, n_raw):
    g, P, U = gen(n), 4096, batch_of_whole_units(H)
    n_pages = pages_of(n, P)
    # dims 0..63 tell the first row from the others, the rest hold a common mean
    vals = torch.randn(n_pages * P, 512, generator=g, device=DEV) * 16 + 240
    vals[:, :64] = 0
    vals[0, :64] = 16.0
    vals[0, 64:] = (1 + torch.rand(448, generator=g, device=DEV)) * torch.randn(448, generator=g, device=DEV).sign()
    codes = vals.to(torch.float8_e4m3fn)
    row_scale = torch.full((n_pages * P,), tail_scale, device=DEV)
    row_scale[0] = head_scale
    q = torch.randn(U, H, 512, generator=g, device=DEV) * (2.0 ** -8 / (240 * max(head_scale, tail_scale)))
    gap = torch.linspace(*gaps, H, device=DEV)
    q[:, :, :64] = (gap / (64 * 16 * head_scale * SCALE))[None, :, None]
    q = q.to(torch.bfloat16)
    raw = torch.randn(U, WINDOW, 512, generator=g, device=DEV).to(torch.float16)
    raw[:, :, :64] = 0
    table = torch.arange(n_pages, device=DEV, dtype=torch.int32).repeat(U, 1)      # all units read the same pages
    out, lse = torch.empty(U, H, 512, dtype=torch.bfloat16, device=DEV), torch.empty(U, H, device=DEV)
    op = cuda_lib.DS4A_OP_PAGED_ATTN_DECODE | (cuda_lib.DS4A_OP_FLAG_128_HEADS if H == 128 else 0)
    ws = torch.empty(cuda_lib.ds4a_workspace_bytes(op, U, 1, n_pages * P, 0), dtype=torch.uint8, device=DEV)
    cuda_lib.ds4a_paged_attn_decode(q, codes.view(torch.uint8).view(n_pages, P, 512), table, ints([n] * U), raw,
                                    ints([n_raw] * U), SCALE, out, lse, ws, row_scale=row_scale.view(n_pages, P))
    assert cuda_lib.ds4a_get_device_status() == (0, 0)
    x = codes[:n].double() * row_scale[:n, None].double()
    for u in (0, U // 2, U - 1):
        check_attn(out[u], lse[u], *attn_reference(q[u], torch.cat((x, raw[u, :n_raw].double())), SCALE))


def test_queries_of_any_size(cuda_lib):
    """q beyond what fp16 holds (65,504; below 2^-14), over FP8 rows alone, as over bf16 rows."""
    g, P, U = gen(3), 64, 3
    codes = (torch.randn(U * P, 512, generator=g, device=DEV) * 100).clamp_(-448, 448).to(torch.float8_e4m3fn)
    for size, s in ((2.0 ** 18, 2.0 ** -26), (2.0 ** -22, 2.0 ** 14)):
        q = (torch.randn(U, 64, 512, generator=g, device=DEV) * size).to(torch.bfloat16)
        row_scale = torch.full((U, P), s, device=DEV)
        out, lse = torch.empty(U, 64, 512, dtype=torch.bfloat16, device=DEV), torch.empty(U, 64, device=DEV)
        ws = torch.empty(cuda_lib.ds4a_workspace_bytes(cuda_lib.DS4A_OP_PAGED_ATTN_DECODE, U, 1, P, 0), dtype=torch.uint8,
                         device=DEV)
        raw = torch.zeros(U, WINDOW, 512, dtype=torch.float16, device=DEV)
        cuda_lib.ds4a_paged_attn_decode(q, codes.view(torch.uint8).view(U, P, 512), ints([[0], [1], [2]]), ints([64, 63, 1]),
                                        raw, ints([0] * U), SCALE, out, lse, ws, row_scale=row_scale)
        assert cuda_lib.ds4a_get_device_status() == (0, 0)
        for u, n in enumerate((64, 63, 1)):
            check_attn(out[u], lse[u], *attn_reference(q[u], codes[u * P:u * P + n].double() * s, SCALE))
