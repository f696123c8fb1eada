"""ds4a_qk_norm_rope against the formula in 64 bits.

Bounds: the fp32 value is off by at most 2^-19 of its pair's size |y_a| + |y_b|
(the sum of squares: 16 products a lane and 5 steps, 21 * 2^-24, halved by the
root; reciprocal root, two products and the rotation's two products and sum a few
2^-23 more; the turn in fp32 2^-25 * 2 pi, sine and cosine 2^-22); its rounding
to 16 bits by at most half a step (bf16 2^-8, fp16 2^-11 of the value, 2^-25 among
fp16's subnormals).  E4M3: half a step is 2^-4 of the value, or 2^-10 scales
among its subnormals."""

import pytest
import torch

from paged_util import DEV, gen, ints, norm_rope_reference

pytestmark = pytest.mark.gpu
EPS = 1e-6
FP32 = 2.0 ** -19


def close(got, ref, size, half, floor=0.0):
    err = FP32 * size
    tol = err + half * (ref.abs() + err) + floor
    d = (got.double() - ref).abs()
    assert (d <= tol).all(), f"off by {float((d / tol.clamp(min=1e-300)).max()):.3f} of the bound"


def freqs(n_rot, theta=10000.0):
    return theta ** (-torch.arange(0, n_rot, 2, dtype=torch.float64, device=DEV) / n_rot)


def inputs(T, H, D, qt, kt, seed=0, pad=0, far=1 << 20):
    g = gen(seed)
    q = (torch.randn(T, H * D + pad, generator=g, device=DEV) * 3).to(qt)[:, :H * D].unflatten(1, (H, D)) if H else None
    k = (torch.randn(T, D + pad, generator=g, device=DEV) * 2).to(kt)[:, :D]
    gq, gk = (1 + 0.2 * torch.randn(D, generator=g, device=DEV) for _ in range(2))
    pos = torch.randint(0, far, (T,), generator=g, device=DEV, dtype=torch.int32)
    return q, k, gq, gk, pos


TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("T,H,D,n_rot,qt,kt,store,pad", [
    (1, 64, 512, 64, "bf16", "bf16", "fp16", 0),
    (1, 1, 512, 16, "fp32", "fp16", "bf16", 0),
    (5, 3, 512, 128, "fp16", "fp32", "bf16", 16),
    (33, 64, 512, 64, "bf16", "fp32", "e4m3", 0),
    (2, 128, 512, 32, "fp32", "bf16", "e4m3", 8),
    (7, 64, 128, 64, "bf16", "fp32", "bf16", 8),
    (1, 1, 128, 128, "fp16", "bf16", "fp16", 0),
    (3, 5, 128, 16, "fp32", "fp16", "bf16", 24),
    (600, 17, 512, 64, "bf16", "bf16", "fp16", 0),      # several heads a warp, the last group short
    (700, 63, 128, 32, "bf16", "bf16", "bf16", 0),      # an odd head count, two rows a warp pass
])
def test_against_the_formula(cuda_lib, T, H, D, n_rot, qt, kt, store, pad, style):
    q, k, gq, gk, pos = inputs(T, H, D, TYPES[qt], TYPES[kt], seed=T + H, pad=pad)
    inv = freqs(n_rot)
    slots = T + 9
    slot = torch.randperm(slots, generator=gen(1), device=DEV)[:T].to(torch.int32)
    q_out = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device=DEV)
    fp8 = store == "e4m3"
    k_out = torch.full((slots, D), 77, dtype=torch.uint8, device=DEV) if fp8 else \
        torch.full((slots, D), 7.0, dtype=TYPES[store], device=DEV)
    scale = torch.full((slots,), 5.0, device=DEV) if fp8 else None
    cuda_lib.ds4a_qk_norm_rope(q, k, pos, inv, EPS, gq, gk, q_out, k_out, k_slot=slot, k_scale=scale, style=style)
    assert cuda_lib.ds4a_get_device_status() == (0, 0)
    ref, size = norm_rope_reference(q, gq, pos, inv, EPS, style)
    close(q_out, ref, size, 2.0 ** -8)
    ref, size = norm_rope_reference(k[:, None], gk, pos, inv, EPS, style)
    ref, size, at = ref[:, 0], size[:, 0], slot.long()
    rest = torch.ones(slots, dtype=torch.bool, device=DEV)
    rest[at] = False
    if fp8:
        amax = ref.abs().amax(-1)
        want = torch.exp2(torch.ceil(torch.log2(amax / 448)))
        border = (amax / want / 448 > 1 - 1e-5) | (amax / want / 448 < 0.5 + 1e-5)   # either side of the border
        assert ((scale[at].double() == want) | border).all()
        got = k_out.view(torch.float8_e4m3fn)[at].double() * scale[at].double()[:, None]
        close(got, ref, size, 2.0 ** -4, floor=2.0 ** -10 * scale[at].double()[:, None])
        assert (k_out[rest] == 77).all() and (scale[rest] == 5).all()
    else:
        close(k_out[at], ref, size, 2.0 ** -8 if store == "bf16" else 2.0 ** -11, 0.0 if store == "bf16" else 2.0 ** -25)
        assert (k_out[rest] == 7).all()


def test_padding_and_slots(cuda_lib):
    """Tokens without a position leave their rows as they were; a negative slot
    stores no key, one past the store is flagged."""
    T, H, D = 6, 4, 512
    q, k, gq, gk, pos = inputs(T, H, D, torch.bfloat16, torch.bfloat16)
    q[1], k[1] = float("nan"), float("inf")
    pos[1] = pos[4] = -1
    slot = ints([3, 0, -1, 9, 1, 2])
    inv = freqs(64)
    q_out = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device=DEV)
    k_out = torch.full((5, D), 7.0, dtype=torch.float16, device=DEV)
    cuda_lib.ds4a_qk_norm_rope(q, k, pos, inv, EPS, gq, gk, q_out, k_out, k_slot=slot)
    assert cuda_lib.ds4a_get_device_status() == (cuda_lib.DS4A_EDEVICE, cuda_lib.DS4A_DEV_BOUNDS)
    live = [0, 2, 3, 5]
    ref, size = norm_rope_reference(q[live], gq, pos[live], inv, EPS, 0)
    close(q_out[live], ref, size, 2.0 ** -8)
    assert (q_out[[1, 4]] == 7).all()
    ref, size = norm_rope_reference(k[[0, 5], None], gk, pos[[0, 5]], inv, EPS, 0)
    close(k_out[[3, 2]], ref[:, 0], size[:, 0], 2.0 ** -11, 2.0 ** -25)
    assert (k_out[[0, 1, 4]] == 7).all()


@pytest.mark.parametrize("theta", [10000.0, 1.5])
def test_far_positions(cuda_lib, theta):
    """Angles up to 2^31 radians: what fp32 products of position and frequency lose."""
    pos = ints([0, 1, 2 ** 20 - 1, 2 ** 24 + 1, 2 ** 30 + 12345, 2 ** 31 - 1])
    q, _, _, _, _ = inputs(6, 2, 512, torch.float32, torch.float32)
    inv = freqs(64, theta)
    q_out = torch.empty(6, 2, 512, dtype=torch.bfloat16, device=DEV)
    cuda_lib.ds4a_qk_norm_rope(q, None, pos, inv, EPS, None, None, q_out, None)
    ref, size = norm_rope_reference(q, None, pos, inv, EPS, 0)
    # the product itself rounds in fp64: 2^-53 of up to 2^31 radians, in both
    close(q_out, ref, size + 2.0 ** 19 * 2.0 ** -21 * size, 2.0 ** -8)


def test_rotation_keeps_dot_products(cuda_lib):
    """q at p and k at p - r meet as they do at r and 0 (the rotation's purpose)."""
    g = gen(3)
    x = torch.randn(1, 1, 512, generator=g, device=DEV)
    y = torch.randn(1, 512, generator=g, device=DEV)
    inv, dots = freqs(64), []
    for p in (7, 1007, 999007):
        for style in (0, 1):
            q_out = torch.empty(1, 1, 512, dtype=torch.bfloat16, device=DEV)
            k_out = torch.empty(1, 512, dtype=torch.bfloat16, device=DEV)
            cuda_lib.ds4a_qk_norm_rope(x, None, ints([p]), inv, EPS, None, None, q_out, None, style=style)
            cuda_lib.ds4a_qk_norm_rope(None, y, ints([p - 7]), inv, EPS, None, None, None, k_out, style=style)
            dots.append((style, float(q_out.double().flatten() @ k_out.double().flatten())))
    bound = 2 * 2.0 ** -8 * 512 * 1.1            # both sides rounded: 2^-8 each of |q| |k| <= 512 (rms 1)
    for style in (0, 1):
        v = [d for s, d in dots if s == style]
        assert max(v) - min(v) <= bound


@pytest.mark.parametrize("row", ["zero", "tiny", "big"])
def test_odd_rows(cuda_lib, row):
    x = torch.randn(1, 1, 512, generator=gen(4), device=DEV) * {"zero": 0.0, "tiny": 1e-12, "big": 1e17}[row]
    q_out = torch.empty(1, 1, 512, dtype=torch.bfloat16, device=DEV)
    k8, scale = torch.empty(1, 512, dtype=torch.uint8, device=DEV), torch.empty(1, device=DEV)
    pos, inv = ints([5]), freqs(64)
    cuda_lib.ds4a_qk_norm_rope(x, x[:, 0], pos, inv, EPS, None, None, q_out, k8, k_scale=scale)
    ref, size = norm_rope_reference(x, None, pos, inv, EPS, 0)
    close(q_out, ref, size, 2.0 ** -8)
    got = k8.view(torch.float8_e4m3fn).double() * scale.double()
    close(got, ref[0], size[0], 2.0 ** -4, floor=2.0 ** -10 * float(scale))
    assert row != "zero" or (float(scale) == 1.0 and not (k8 & 127).any())      # codes of +-0


@pytest.mark.parametrize("D,H", [(512, 64), (512, 7), (128, 64), (128, 9)])
def test_q_in_place(cuda_lib, D, H):
    q, _, gq, _, pos = inputs(301, H, D, torch.bfloat16, torch.bfloat16)
    inv, other = freqs(64), torch.empty(301, H, D, dtype=torch.bfloat16, device=DEV)
    q = q.contiguous()
    cuda_lib.ds4a_qk_norm_rope(q, None, pos, inv, EPS, gq, None, other, None)
    cuda_lib.ds4a_qk_norm_rope(q, None, pos, inv, EPS, gq, None, q, None)
    assert torch.equal(q, other)


def test_no_token(cuda_lib):
    e = torch.empty
    cuda_lib.ds4a_qk_norm_rope(e(0, 64, 512, dtype=torch.bfloat16, device=DEV), e(0, 512, device=DEV), ints([]), freqs(64),
                               EPS, None, None, e(0, 64, 512, dtype=torch.bfloat16, device=DEV),
                               e(4, 512, dtype=torch.float16, device=DEV))
    assert cuda_lib.ds4a_get_device_status() == (0, 0)


def test_captured_and_on_two_streams(cuda_lib):
    q, k, gq, gk, pos = inputs(40, 64, 512, torch.bfloat16, torch.bfloat16)
    inv = freqs(64)
    outs = [(torch.empty(40, 64, 512, dtype=torch.bfloat16, device=DEV), torch.empty(40, 512, dtype=torch.bfloat16, device=DEV))
            for _ in range(3)]

    def go(i, stream=None):
        cuda_lib.ds4a_qk_norm_rope(q, k, pos, inv, EPS, gq, gk, *outs[i], stream=stream)
    go(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    go(1, side)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        go(2)
    pos.add_(1)
    graph.replay()
    ref, size = norm_rope_reference(q, gq, pos, inv, EPS, 0)
    close(outs[2][0], ref, size, 2.0 ** -8)
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_rejects_other_tensors(cuda_lib):
    q, k, gq, gk, pos = inputs(4, 64, 512, torch.bfloat16, torch.bfloat16)
    inv = freqs(64)
    qo, ko = torch.empty_like(q).contiguous(), torch.empty_like(k).contiguous()
    good = dict(q=q, k=k, pos=pos, inv_freq=inv, eps=EPS, q_weight=gq, k_weight=gk, q_out=qo, k_out=ko)
    for change in (dict(q=q.double()), dict(q=q.cpu()), dict(q=q[:, :, :256]), dict(q=q.transpose(0, 1)), dict(q_out=qo.float()),
                   dict(q_out=qo[:, :32]), dict(k=k.int()), dict(k=k[:3]), dict(k_out=ko.double()), dict(k_out=ko[:, :256]),
                   dict(k_out=None), dict(pos=pos.long()), dict(pos=pos[:3]), dict(inv_freq=inv.float()), dict(q_weight=gq[:8]),
                   dict(k_weight=gk.half()), dict(q=None, k=None), dict(k_out=torch.empty(4, 512, dtype=torch.uint8, device=DEV))):
        with pytest.raises(ValueError):
            cuda_lib.ds4a_qk_norm_rope(**dict(good, **change))
    for change in (dict(k_out=ko[:3]), dict(inv_freq=freqs(64)[:5]), dict(eps=0.0)):
        with pytest.raises(cuda_lib.Ds4aError):
            cuda_lib.ds4a_qk_norm_rope(**dict(good, **change))
