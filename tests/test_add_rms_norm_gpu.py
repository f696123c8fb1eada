"""ds4a_add_rms_norm against the formula in 64 bits.

Bounds: h = x + res is one fp32 sum (2^-24 of itself).  The sum of squares adds at
most 40 roundings along any path (32 of a thread, the butterfly, the warps), its
root halves their weight, rsqrt and three products add 8 more: y is off by less than
2^-18 of itself before its one rounding, half a step of its type."""
import pytest
import torch

from paged_util import DEV, gen, ints

pytestmark = pytest.mark.gpu
EPS = 1e-6
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
FP32 = 2.0 ** -18
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def reference(x, res, weight):
    h = x.double() + (res.double() if res is not None else 0.0)
    y = h / ((h * h).mean(-1, keepdim=True) + EPS).sqrt()
    return h, y * (weight.double() if weight is not None else 1.0)


def check_value(got, ref, rel):
    half = HALF[got.dtype]
    floor = 2.0 ** -25 if got.dtype == HF else 1e-38          # half a subnormal step
    tol = rel * ref.abs() + half * (1 + rel) * ref.abs() + floor
    assert ((got.double() - ref).abs() <= tol).all()


def check_codes(codes, scales, y, group, pow2):
    T, D = y.shape
    group = group or D
    G = -(-D // group)
    pad = torch.zeros(T, G * group, dtype=torch.float64, device=y.device)
    pad[:, :D] = y
    amax = pad.view(T, G, group).abs().amax(-1)
    s = scales.double().view(T, G)
    if pow2:
        assert (torch.frexp(scales)[0] == 0.5).all()
        some = amax > 0
        assert (amax <= 448 * s * (1 + FP32))[some].all()
        assert (amax >= 224 * s * (1 - FP32))[some & (s > 2.0 ** -126)].all()
    else:
        want = torch.where(amax > 0, (amax / 448).clamp(min=2.0 ** -126), 1.0)
        assert ((s - want).abs() <= (FP32 + 2.0 ** -22) * want).all()
    wide = s.repeat_interleave(group, 1)[:, :D]
    v = codes.view(torch.float8_e4m3fn).double() * wide
    # half a step of e4m3 (2^-4 of a normal value, 2^-10 of the scale below), a scale in fp32
    tol = (2.0 ** -4 + FP32) * y.abs() + FP32 * y.abs() + 2.0 ** -10 * wide * (1 + FP32)
    assert ((v - y).abs() <= tol).all()


def rows(g, T, D, dtype, spread, pad=0):
    full = torch.randn(T, D + pad, generator=g, device=DEV) * spread
    return full.to(dtype)[:, :D]


@pytest.mark.parametrize("T,D", [(1, 8), (1, 4096), (3, 16384), (5, 40), (1, 16376), (700, 128), (333, 1000), (400, 8200),
                                 (17, 504), (1000, 512), (310, 16384), (2000, 1024)])
@pytest.mark.parametrize("xt,rt,ot,group,pow2", [(BF, BF, BF, 128, True), (BF, F32, None, 128, False), (F32, F32, F32, 32, False),
                                                 (HF, None, HF, 64, True), (F32, BF, BF, 0, True), (BF, HF, F32, 0, False),
                                                 (BF, None, BF, None, True)])
def test_rows(cuda_lib, T, D, xt, rt, ot, group, pow2):
    g = gen(T * D)
    x = rows(g, T, D, xt, 3.0, pad=8)
    res = rows(g, T, D, rt, 5.0, pad=16) if rt else None
    weight = 1 + 0.2 * torch.randn(D, generator=g, device=DEV) if T % 2 else None
    res_out = torch.zeros(T, D, dtype=rt, device=DEV) if rt else None
    out = torch.zeros(T, D, dtype=ot, device=DEV) if ot else None
    codes = scales = None
    if group is not None:
        codes = torch.zeros(T, D, dtype=torch.uint8, device=DEV)
        scales = torch.zeros(T, -(-D // group) if group else 1, device=DEV)
    cuda_lib.ds4a_add_rms_norm(x, weight, EPS, out=out, residual=res, res_out=res_out, codes=codes, scales=scales,
                               group=group or 0, scale_style=0 if pow2 else 1)
    assert cuda_lib.ds4a_get_device_status() == (0, 0)
    h, y = reference(x, res, weight)
    if rt:
        check_value(res_out, h, 2.0 ** -24)
    if ot:
        check_value(out, y, FP32)
    if group is not None:
        check_codes(codes, scales, y, group, pow2)


def test_residual_in_place_and_a_padded_batch(cuda_lib):
    T, D = 50, 2048
    g = gen(1)
    x, res, w = rows(g, T, D, BF, 1.0), rows(g, T, D, BF, 2.0).contiguous(), torch.rand(D, generator=g, device=DEV)
    for live in (0, 1, 37, 50):
        r = res.clone()
        out, codes, scales = torch.full((T, D), 7.0, device=DEV), torch.full((T, D), 9, dtype=torch.uint8, device=DEV), \
            torch.full((T, 16), 7.0, device=DEV)
        cuda_lib.ds4a_add_rms_norm(x, w, EPS, out=out, residual=r, res_out=r, codes=codes, scales=scales, n_live=ints([live]))
        h, y = reference(x, res, w)
        check_value(r[:live], h[:live], 2.0 ** -24)
        check_value(out[:live], y[:live], FP32)
        check_codes(codes[:live], scales[:live], y[:live], 128, True)
        assert torch.equal(r[live:], res[live:]) and (out[live:] == 7).all() and (codes[live:] == 9).all()
        assert (scales[live:] == 7).all()
    assert cuda_lib.ds4a_get_device_status() == (0, 0)
    for bad, rows_done in ((-1, 0), (51, 50)):
        out = torch.full((T, D), 7.0, device=DEV)
        cuda_lib.ds4a_add_rms_norm(x, w, EPS, out=out, n_live=ints([bad]))
        assert cuda_lib.ds4a_get_device_status() == (cuda_lib.DS4A_EDEVICE, cuda_lib.DS4A_DEV_BOUNDS)
        assert (out[rows_done:] == 7).all() and (out[:rows_done] != 7).any(-1).all()


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("pow2", [True, False])
def test_special_values(cuda_lib, group, pow2):
    """Zeros, a NaN, an infinity, tiny and huge rows."""
    D = 512
    x = torch.randn(7, D, generator=gen(2), device=DEV)
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 300] = float("inf")
    x[3] *= 1e-25
    x[4] *= 1e25                                    # the squares pass the fp32 range
    x[5, 128:256] = 0
    codes, scales = torch.empty(7, D, dtype=torch.uint8, device=DEV), torch.empty(7, 4 if group else 1, device=DEV)
    out = torch.empty(7, D, device=DEV)
    cuda_lib.ds4a_add_rms_norm(x, None, EPS, out=out, codes=codes, scales=scales, group=group, scale_style=0 if pow2 else 1)
    assert cuda_lib.ds4a_get_device_status() == (0, 0)
    v = codes.view(torch.float8_e4m3fn).float()
    assert (out[0] == 0).all() and (v[0] == 0).all() and (scales[0] == 1).all()
    assert out[1].isnan().all() and v[1].isnan().all() and (scales[1] == 1).all()
    assert out[2, 300].isnan() and (out[2, :300] == 0).all()           # inf * 0
    _, y = reference(x, None, None)
    check_value(out[[3, 5, 6]], y[[3, 5, 6]], FP32)
    check_codes(codes[[3, 5, 6]], scales[[3, 5, 6]], y[[3, 5, 6]], group, pow2)
    assert (out[4] == 0).all() and (v[4] == 0).all()


def test_same_codes_as_the_row_store(cuda_lib):
    """A power of two per row of 512 is the FP8 row store's round trip."""
    x = torch.randn(300, 512, generator=gen(3), device=DEV) * torch.logspace(-8, 8, 300, device=DEV)[:, None]
    y, c1, s1 = torch.empty_like(x), torch.empty(300, 512, dtype=torch.uint8, device=DEV), torch.empty(300, 1, device=DEV)
    cuda_lib.ds4a_add_rms_norm(x, None, EPS, out=y, codes=c1, scales=s1, group=0)
    c2, s2 = torch.empty_like(c1), torch.empty(300, device=DEV)
    cuda_lib.ds4a_rows_to_fp8(y, c2, s2)
    assert torch.equal(c1, c2) and torch.equal(s1[:, 0], s2)


def test_captured_on_another_stream(cuda_lib):
    T, D = 64, 4096
    g = gen(4)
    x, res, w = rows(g, T, D, BF, 1.0), rows(g, T, D, F32, 1.0).contiguous(), torch.rand(D, generator=g, device=DEV)
    out, n = torch.zeros(T, D, dtype=BF, device=DEV), ints([T])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    cuda_lib.ds4a_add_rms_norm(x, w, EPS, out=out, residual=res, n_live=n, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        cuda_lib.ds4a_add_rms_norm(x, w, EPS, out=out, residual=res, res_out=res, n_live=n)
    start = res.clone()
    for live in (64, 3):
        n.fill_(live)
        res.copy_(start)
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        h, y = reference(x, start, w)
        check_value(out[:live], y[:live], FP32)
        assert (out[live:] == 0).all() and torch.equal(res[live:], start[live:])


def test_no_row(cuda_lib):
    x = torch.empty(0, 512, dtype=BF, device=DEV)
    cuda_lib.ds4a_add_rms_norm(x, None, EPS, out=torch.empty_like(x))
    assert cuda_lib.ds4a_get_device_status() == (0, 0)


def test_rejects_other_tensors(cuda_lib):
    x, w = torch.zeros(4, 256, dtype=BF, device=DEV), torch.ones(256, device=DEV)
    out, codes, scales = torch.empty_like(x), torch.empty(4, 256, dtype=torch.uint8, device=DEV), torch.empty(4, 2, device=DEV)
    good = dict(x=x, weight=w, eps=EPS, out=out, residual=x, res_out=torch.empty_like(x), codes=codes, scales=scales)
    for change in (dict(x=x.cpu()), dict(x=x.to(torch.float64)), dict(x=x[None]), dict(x=x[:, ::2]), dict(weight=w.half()),
                   dict(weight=w[:128]), dict(out=torch.empty(4, 512, dtype=BF, device=DEV)[:, :256]), dict(out=codes),
                   dict(residual=None), dict(residual=x[:2]), dict(res_out=torch.empty(4, 256, device=DEV)),
                   dict(codes=None), dict(scales=scales[:, :1]), dict(scales=scales.half()), dict(n_live=torch.zeros(1, device=DEV)),
                   dict(codes=codes[:2]), dict(group=64)):
        with pytest.raises(ValueError):
            cuda_lib.ds4a_add_rms_norm(**dict(good, **change))
    with pytest.raises(cuda_lib.Ds4aError):
        cuda_lib.ds4a_add_rms_norm(x, w, EPS)
