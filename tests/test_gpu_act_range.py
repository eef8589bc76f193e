"""The 4-bit entries where scales saturate or vanish and where global scales are extreme, on the GPU."""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_packed_gb300 as wqp

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.bfloat16, torch.float16, torch.float32]
E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
MIDDLES = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0])


def unpack4(codes):
    c = codes.cpu()
    return torch.stack((c & 15, c >> 4), 2).view(c.shape[0], -1)


def codes_of(x, d):
    """E2M1 codes of the FP32 quotients x / d (correctly rounded on the host), to nearest even, saturating."""
    q = x / d
    a = q.abs()
    mag = (a > .25).int() + (a >= .75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
    return (mag + 8 * torch.signbit(q)).to(torch.uint8)


def near_middles(d, groups, dtype, seed):
    """[groups, 16] values at, just below and just above a middle between two codes times d, of either sign."""
    g = torch.Generator().manual_seed(seed)
    v = (MIDDLES[torch.randint(0, 7, (groups, 16), generator=g)].double() * float(d)).to(dtype)
    bits = torch.int32 if dtype is torch.float32 else torch.int16
    v = (v.view(bits) + torch.randint(-1, 2, (groups, 16), generator=g).to(bits)).view(dtype)
    return torch.where(torch.rand((groups, 16), generator=g) < 0.5, -v, v)


def saturating(dtype, g, over):
    """(d, amax) of groups whose amax / (6 g) is `over` times the largest scale."""
    d = float(torch.tensor(448.0) * torch.tensor(g))
    return d, torch.tensor(over * 6 * d, dtype=torch.float64).to(dtype)


def in_range(dtype, g, over):
    d, amax = saturating(dtype, g, over)
    return bool(amax.isfinite()) and float(amax) > 5.2 * d and bool(torch.tensor(d / 4).to(dtype) > 0)


# Global scales with few and with many bits, tiny and large; what of them the type can hold.
@pytest.mark.parametrize("dtype,g,over", [
    (t, g, over) for t in TYPES for g in [0.53125, 0.00059581938, 1.0, 0.3, 1.1 * 2.0 ** -20, 1.37 * 2.0 ** -100, 1.9 * 2.0 ** 60]
    for over in [1.0, 1.0004, 1.7, 1000.0, 2.0 ** 95, 2.0 ** 103, 2.0 ** 120] if in_range(t, g, over)])
def test_w4_quantize_rounds_the_quotient_in_every_group(dtype, g, over):
    """Elements around the middles between two codes, of groups at and beyond the largest scale."""
    g, groups = float(torch.tensor(g)), 512
    d, amax = saturating(dtype, g, over)
    x = near_middles(d, groups, dtype, seed=int(over) % 97 + 1)
    x[:, 3] = torch.where(torch.arange(groups) % 2 == 0, amax, -amax)
    codes, scales = wqp.w4_quantize(x.view(8, -1).to(DEV), g)
    assert (scales == 0x7E).all()
    assert torch.equal(unpack4(codes).view(groups, 16), codes_of(x.float(), torch.tensor(d)))


def test_w4_quantize_calibrated_global_scale():
    """g = amax / (6 * 448), as a calibration gives it: in FP32 the largest group then often passes 448 by a little."""
    groups, hit = 64, 0
    for seed in range(40):
        amax = float((1 + torch.rand(1, generator=torch.Generator().manual_seed(seed))).bfloat16())
        g = float(torch.tensor(amax / (6 * 448)))
        d = torch.tensor(448.0) * torch.tensor(g)
        x = near_middles(d, groups, torch.bfloat16, seed)
        x[:, 0] = amax
        codes, scales = wqp.w4_quantize(x.view(1, -1).to(DEV), g)
        assert (scales == 0x7E).all()
        assert torch.equal(unpack4(codes).view(groups, 16), codes_of(x.float(), d))
        hit += bool(torch.tensor(amax) / (torch.tensor(6.0) * torch.tensor(g)) > 448)
    assert hit


@pytest.mark.parametrize("dtype", TYPES)
def test_w4_quantize_codes_under_a_zero_scale_are_zero(dtype):
    """Elements of either sign in groups whose scale rounds to nothing."""
    x = torch.zeros(4, 128)
    x[1] = 2.0 ** -14
    x[2] = -(2.0 ** -14)
    x[3, ::3] = -0.0
    x[3, 1::3] = -(2.0 ** -15)
    codes, scales = wqp.w4_quantize(x.to(dtype).to(DEV), 1.0)
    assert not scales.any() and not codes.any()


# ---------------------------------------------------------------- products
def operand(R, K, lo, hi, seed):
    """Every code, scale codes lo..hi, and the values without a global scale; one of several rows is zeros."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    codes = torch.randint(0, 256, (R, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    if R > 1:
        codes[R // 2] = 0
    scales = torch.randint(lo, hi + 1, (R, K // 16), generator=g, device=DEV, dtype=torch.uint8)
    v = E2M1.to(DEV)[torch.stack((codes & 15, codes >> 4), 2).view(R, K).long()]
    return codes, scales, (v.view(R, -1, 16) * scales.view(torch.float8_e4m3fn).double().unsqueeze(2)).view(R, K)


# (scale codes, a_global, w_global): products of the two that FP32 holds only as 0, with few bits, or as infinity, beside
# ones that it holds.
RANGES = {
    "vanishing": ((0x70, 0x7E), 1.1 * 2.0 ** -78, 1.3 * 2.0 ** -74), "few bits": ((0x70, 0x7E), 1.7 * 2.0 ** -70, -1.9 * 2.0 ** -77),
    "one subnormal": ((0x70, 0x7E), 1.37 * 2.0 ** -127, 2.0 ** -10), "infinite": ((0x01, 0x08), 1.1 * 2.0 ** 64, 1.2 * 2.0 ** 64),
    "far infinite": ((0x01, 0x08), -1.5 * 2.0 ** 90, 1.25 * 2.0 ** 100), "opposite": ((0x30, 0x40), 1.1 * 2.0 ** 100, 1.2 * 2.0 ** -100),
}


# Few rows with and without split K; many rows of either tile orientation.
@pytest.mark.parametrize("M,N,K", [(1, 300, 768), (20, 200, 5120), (64, 20000, 256), (130, 20000, 256), (300, 640, 768), (128, 34816, 512)])
@pytest.mark.parametrize("name", sorted(RANGES))
def test_w4a4_extreme_global_scales(name, M, N, K):
    """C = a_global * w_global * sum wherever that is in BF16's range: zeros stay zeros, and what passes the range
    becomes infinite."""
    (lo, hi), ga, gw = RANGES[name]
    ga, gw = float(torch.tensor(ga)), float(torch.tensor(gw))
    a, sa, av = operand(M, K, lo, hi, M + N)
    w, sw, wv = operand(N, K, lo, hi, M + N + 1)
    C = wqp.w4a4_gemm(a, sa, w, sw, N, K, ga, gw).double()
    ref = (av @ wv.t()) * (ga * gw)
    off = (K / 32 + 16) * 2.0 ** -22 * (av.abs() @ wv.abs().t()) * abs(ga * gw)      # of the sum
    # BF16 ends at 255 * 2^120 (what rounds beyond is infinite); 2^-134 is half its least step.
    top = 255.5 * 2.0 ** 120
    inside = ref.abs() + off < top
    assert ((C - ref).abs() <= 2.0 ** -8 * ref.abs() + 2 * off + 2.0 ** -134)[inside].all()
    beyond = ref.abs() - off > top
    assert (C == torch.sign(ref) * float("inf"))[beyond].all()
    assert not C.isnan().any() and (C[:, N // 2] == 0).all() and (M == 1 or (C[M // 2] == 0).all())
    assert C.any() and (inside.all() or name == "far infinite")
    assert wqp.get_device_error() == 0
