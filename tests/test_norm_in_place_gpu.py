"""The residual norm in place of its inputs, and between the halves of one buffer: the same
bits as apart."""
import pytest
import torch

from paged_util import DEV, gen, ints

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def norm(lib, x, w, res, res_out, out, codes=True, n_live=None):
    T, D = x.shape
    c = s = None
    if codes:
        c, s = torch.full((T, D), 9, dtype=torch.uint8, device=DEV), torch.full((T, -(-D // 128)), 9.0, device=DEV)
    lib.ds4a_add_rms_norm(x, w, 1e-6, out=out, residual=res, res_out=res_out, codes=c, scales=s, n_live=n_live)
    assert lib.ds4a_get_device_status() == (0, 0)
    return c, s


@pytest.mark.parametrize("T,D", [(1, 4096), (3, 40), (500, 1000), (400, 8200), (700, 4096)])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_in_place(cuda_lib, T, D, dtype):
    g = gen(T + D)
    x, res = (torch.randn(T, D, generator=g, device=DEV).to(dtype) for _ in range(2))
    w, live = torch.randn(D, generator=g, device=DEV), ints([T - T // 3])
    h, y = x.clone(), x.clone()                      # (rows behind the live ones stay what they were)
    c0, s0 = norm(cuda_lib, x, w, res, h, y, n_live=live)
    h2, y2 = res.clone(), res.clone()
    norm(cuda_lib, x, w, res, h2, y2, n_live=live)
    n = T - T // 3
    # out is x
    a, b = x.clone(), res.clone()
    c, s = norm(cuda_lib, a, w, b, b, a, n_live=live)
    assert torch.equal(a, y) and torch.equal(b, h2) and torch.equal(c, c0) and torch.equal(s, s0)
    # res_out is x, out is res
    a, b = x.clone(), res.clone()
    c, s = norm(cuda_lib, a, w, b, a, b, n_live=live)
    assert torch.equal(a, h) and torch.equal(b, y2) and torch.equal(c, c0) and torch.equal(s, s0)
    # out is x without a residual
    a, want = x.clone(), torch.empty_like(x)
    norm(cuda_lib, x, w, None, None, want, codes=False)
    norm(cuda_lib, a, w, None, None, a, codes=False)
    assert torch.equal(a, want) and not torch.equal(a[:n], x[:n])


@pytest.mark.parametrize("T,D", [(5, 512), (600, 2048)])
def test_halves_of_one_buffer(cuda_lib, T, D):
    g = gen(D)
    both = torch.randn(T, 3 * D, generator=g, device=DEV).to(BF)
    x, res, to = both[:, :D], both[:, D:2 * D], both[:, 2 * D:]
    want, out0, out = torch.empty(T, D, dtype=BF, device=DEV), torch.empty(T, D, dtype=BF, device=DEV), torch.empty(T, D, dtype=BF, device=DEV)
    norm(cuda_lib, x.contiguous(), None, res.contiguous(), want, out0)
    keep = both[:, :2 * D].clone()
    norm(cuda_lib, x, None, res, to, out)
    assert torch.equal(to, want) and torch.equal(out, out0) and torch.equal(both[:, :2 * D], keep)
    norm(cuda_lib, x, None, res, x, out)             # res_out is x, rows apart
    assert torch.equal(x, want) and torch.equal(out, out0)


def test_refuses_overlaps(cuda_lib):
    x = torch.zeros(9, 512, dtype=BF, device=DEV)
    r = torch.zeros(8, 512, dtype=BF, device=DEV)
    codes, scales = torch.zeros(8, 512, dtype=torch.uint8, device=DEV), torch.zeros(8, 4, device=DEV)
    good = dict(x=x[:8], weight=None, eps=1e-6, residual=r, res_out=r, codes=codes, scales=scales)
    for change in (dict(out=x[1:]), dict(out=r), dict(res_out=x[1:]),
                   dict(codes=x[:8].view(torch.uint8).view(-1)[:8 * 512].view(8, 512))):
        with pytest.raises(cuda_lib.Ds4aError):
            cuda_lib.ds4a_add_rms_norm(**dict(good, **change))
    assert cuda_lib.ds4a_get_device_status() == (0, 0)
