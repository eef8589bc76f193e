"""The 4-bit quantiser where scales saturate or vanish, on the GPU."""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_packed_gb300 as wqp

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.bfloat16, torch.float16, torch.float32]
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
