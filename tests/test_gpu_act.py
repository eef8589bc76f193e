"""The quantised-activation entries on the GPU against plain 64-bit forms.

Tolerances, each from the arithmetic alone (u = 2^-24):

* Quantisers. The scale is the nearest code (or FP32 value) to its quotient,
  and each code the nearest to its own, up to the rounding of the FP32 quotient
  they are taken from: a relative 4 u.
* Norm. The sum of squares has positive terms, so n additions in any order are
  off by at most n u of it, with n <= K / 1024 + 64 along any path of the
  kernels; the root halves that, and the remaining operations add 8 u. Rounding
  to the output's type is monotonous, so an output lies between the roundings of
  that interval's ends.
* Products. All products are exact in FP32. A sum of K of them, in steps of at
  least 32 per MMA, each step rounded or cut to 2^-23 of the largest partial sum,
  is off by at most (K / 32 + 16) 2^-22 S, S the sum of magnitudes (the 8-bit
  path's FP32 factor adds 4 u per block, inside that). BF16 output adds 2^-8.
  Where all partial sums are integers below 2^24 the result is the exact one.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import weight_only_quantized_packed_gb300 as wqp

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float16, torch.float32]
E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rows(M, K, dtype, pad, seed, scale=1.0):
    """Normal rows with some large channels, K + pad apart."""
    g = gen(seed)
    buf = torch.full((M, K + pad), 77.0, dtype=dtype, device=DEV)
    x = torch.randn((M, K), generator=g, device=DEV) * scale
    x *= torch.where(torch.rand(K, generator=g, device=DEV) < 0.02, 12.0, 1.0)
    buf[:, :K] = x.to(dtype)
    return buf[:, :K]


def unpack4(codes):
    c = codes.cpu()
    return torch.stack((c & 15, c >> 4), 2).view(c.shape[0], -1)


def e4m3(codes):
    return codes.cpu().view(torch.float8_e4m3fn).double()


E4M3_ALL = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()     # 0 .. 448


def assert_nearest(v, got, values, rel):
    """got is a value of `values` (sorted) nearest to v, up to rel of v; v saturates at the largest."""
    v = v.clamp(max=values[-1])
    i = torch.searchsorted(values, v.contiguous()).clamp(max=len(values) - 1)
    best = torch.minimum((values[i] - v).abs(), (values[(i - 1).clamp(min=0)] - v).abs())
    assert ((got - v).abs() <= best + rel * v.abs()).all()


# ---------------------------------------------------------------- quantisers
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,pad", [(1, 128, 0), (3, 384, 8), (17, 5120, 0), (301, 640, 40), (2, 65536, 0), (1, 256, 24)])
@pytest.mark.parametrize("g", [1.0, 0.25, 2.0 ** -9])
def test_w4_quantize(dtype, M, K, pad, g):
    x = rows(M, K, dtype, pad, seed=M + K)
    codes, scales = wqp.w4_quantize(x, g)
    assert codes.shape == (M, K // 2) and scales.shape == (M, K // 16)
    x64 = x.double().cpu().view(M, -1, 16)
    s = e4m3(scales)
    assert_nearest(x64.abs().amax(2) / (6 * g), s, E4M3_ALL, 4 * U)
    d = (s * g).unsqueeze(2)
    v = E2M1[unpack4(codes).long()].view(M, -1, 16)
    live = (d > 0).expand_as(v)
    q = torch.where(live, x64 / torch.where(d > 0, d, 1.0), 0.0)
    assert (v[~live] == 0).all()
    assert_nearest(q.abs(), v.abs(), E2M1[:8], 4 * U)
    assert ((v == 0) | (torch.sign(v) == torch.sign(x64))).all()
    # The format is the W4A16 one: the framework's own unpacking agrees.
    back = wqp.w4a16_dequant(codes, scales, M, K, g).double().cpu().view(M, -1, 16)
    assert torch.equal(back, v * d)


@pytest.mark.parametrize("dtype", TYPES)
def test_w4_quantize_ties_go_to_even(dtype):
    """Every scale mantissa with elements on the middles between codes: the quotients are exact."""
    middles = [(.25, 0), (.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6)]
    groups, want, scale = [], [], []
    for e in (-5, 0, 4):
        for m in range(8, 16):
            s = m / 8 * 2.0 ** e
            vals = [6.0 * s, -6.0 * s] + [b * s for b, _ in middles] + [-b * s for b, _ in middles]
            groups.append(vals)
            want.append([7, 15] + [c for _, c in middles] + [c | 8 for _, c in middles])
            scale.append(s)
    K = 16 * len(groups)
    x = torch.tensor(groups, dtype=torch.float64).view(1, K)
    assert torch.equal(x.to(dtype).double(), x)
    codes, scales = wqp.w4_quantize(x.to(dtype).to(DEV), 1.0)
    assert torch.equal(e4m3(scales).view(-1), torch.tensor(scale, dtype=torch.float64))
    assert torch.equal(E2M1[unpack4(codes).long()].view(-1), E2M1[torch.tensor(want).view(-1)])


@pytest.mark.parametrize("dtype", TYPES)
def test_w4_quantize_special_groups(dtype):
    inf, nan = float("inf"), float("nan")
    x = torch.zeros(1, 128, dtype=torch.float32)
    x[0, 16] = nan
    x[0, 33:36] = torch.tensor([inf, 1.0, -2.0])
    x[0, 48] = -inf
    x[0, 64:68] = torch.tensor([60000.0, -60000.0, 1.0, -1.0])      # scale saturates at 448
    x[0, 80] = 2.0 ** -14                                           # scale rounds to nothing
    x[0, 96:98] = torch.tensor([6 * 2.0 ** -9, -(2.0 ** -9)])       # the least scale
    codes, scales = wqp.w4_quantize(x.to(dtype).to(DEV), 1.0)
    c, s = unpack4(codes).view(8, 16), scales.cpu().view(-1).tolist()
    assert s[0] == 0 and s[1] == s[2] == s[3] == 0x7F and s[4] == 0x7E and s[5] == 0 and s[6] == 1 and s[7] == 0
    assert not c[:4].any()
    assert c[4, :4].tolist() == [7, 15, 0, 8] and not c[4, 4:].any()
    assert not (c[5] & 7).any() and c[6, :2].tolist() == [7, 10]
    assert wqp.w4a16_dequant(codes, scales, 1, 128, 1.0).isnan().view(8, 16).any(1).tolist() == [False, True, True, True] + [False] * 4


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,pad", [(1, 128, 0), (3, 384, 8), (17, 5120, 0), (301, 640, 40), (2, 65536, 0), (1, 256, 24)])
def test_a8_quantize(dtype, M, K, pad):
    x = rows(M, K, dtype, pad, seed=M + K + 1)
    codes, scales = wqp.a8_quantize(x)
    x64 = x.double().cpu().view(M, -1, 128)
    amax = x64.abs().amax(2)
    s = scales.double().cpu()
    assert ((s - amax / 448).abs() <= U * s).all()
    v = e4m3(codes).view(M, -1, 128)
    q = x64 * (448 / amax).unsqueeze(2)
    assert_nearest(q.abs(), v.abs(), E4M3_ALL, 4 * U)
    assert ((v == 0) | (torch.sign(v) == torch.sign(x64))).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_a8_quantize_special_groups(dtype):
    x = torch.zeros(5, 128)
    x[1, 7] = float("nan")
    x[2, 8] = float("-inf")
    x[3, 9] = 2.0 ** -24
    x[4, :2] = torch.tensor([-448.0, 1.0])
    codes, scales = wqp.a8_quantize(x.to(dtype).to(DEV))
    v, s = e4m3(codes), scales.cpu()[:, 0]
    assert not v[0].any() and float(s[0]) == float(np.float32(2.0 ** -100) / np.float32(448))
    assert s[1].isnan() and s[2].isnan() and v[1].isnan().all() and v[2].isnan().all()
    assert v[3, 9] == 448 and abs(float(s[3]) - 2.0 ** -24 / 448) <= U * float(s[3])
    assert s[4] == 1 and v[4, :2].tolist() == [-448, 1]


# ---------------------------------------------------------------- norm
def assert_rounded(got, ref, off):
    """got is a rounding, to its type, of a value within a relative off of ref."""
    lo, hi = (ref - off * ref.abs()).to(got.dtype), (ref + off * ref.abs()).to(got.dtype)
    got = got.cpu()
    assert ((lo <= got) & (got <= hi)).all()


def norm64(x, r, w, eps):
    h = x.double().cpu() + (0 if r is None else r.double().cpu())
    return h, h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * w.double().cpu()


NORMS = [(1, 128, 0), (700, 128, 0), (5, 384, 8), (2, 1024, 40), (1, 5120, 0), (700, 5120, 0), (650, 4224, 8), (3, 17408, 0),
         (611, 8192, 0), (2, 65536, 0)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("M,K,pad", NORMS)
def test_rms_norm(dtype, residual, M, K, pad):
    x, w = rows(M, K, dtype, pad, 3 * M + K), (1 + 0.2 * torch.randn(K, generator=gen(5), device=DEV)).to(dtype)
    r = rows(M, K, dtype, pad, 7 * M + K, scale=3.0) if residual else None
    eps = 1e-5
    h64, y64 = norm64(x, r, w, eps)
    off = ((K / 1024 + 64) / 2 + 8) * U
    y, h = wqp.rms_norm(x, w, eps, residual=r)
    assert_rounded(y, y64, off)
    codes, scales, h8 = wqp.rms_norm_a8(x, w, eps, residual=r)
    s = scales.double().cpu()
    amax = y64.view(M, -1, 128).abs().amax(2)
    assert ((s - amax / 448).abs() <= (off + 2 * U) * s).all()
    v = e4m3(codes).view(M, -1, 128)
    q = y64.view(M, -1, 128) / s.unsqueeze(2)
    assert_nearest(q.abs(), v.abs(), E4M3_ALL, 2 * off + 4 * U)
    if residual:
        assert torch.equal(h, h8)
        assert_rounded(h, h64, U)
    else:
        assert h is None and h8 is None


@pytest.mark.parametrize("M,K", [(3, 640), (700, 5120), (2, 40960)])
def test_rms_norm_in_place_and_canaries(M, K):
    """The sum written over the residual, y over x, in rows with a pitch: the bytes between rows stay."""
    w = torch.ones(K, dtype=torch.bfloat16, device=DEV)
    x, r = rows(M, K, torch.bfloat16, 16, 1), rows(M, K, torch.bfloat16, 24, 2)
    want_y, want_h = wqp.rms_norm(x, w, 1e-6, residual=r)
    want8 = wqp.rms_norm_a8(x, w, 1e-6, residual=r)
    r2 = rows(M, K, torch.bfloat16, 24, 2)
    c, s, h = wqp.rms_norm_a8(x, w, 1e-6, residual=r2, residual_out=r2)
    assert h is r2 and torch.equal(r2, want_h) and torch.equal(c, want8[0]) and torch.equal(s, want8[1])
    y, h = wqp.rms_norm(x, w, 1e-6, residual=r, residual_out=r, out=x)
    assert torch.equal(y, want_y) and torch.equal(r, want_h)
    for t, pad in ((x, 16), (r, 24), (r2, 24)):
        assert (torch.as_strided(t, (M, pad), (t.stride(0), 1), t.storage_offset() + K) == 77).all()


@pytest.mark.parametrize("K", [128, 5120, 65536])
def test_rms_norm_special_rows(K):
    x = torch.randn(5, K, generator=gen(9), device=DEV).bfloat16()
    x[1] = 0
    x[2, 3] = float("inf")
    x[3, 100] = float("nan")
    w = torch.ones(K, dtype=torch.bfloat16, device=DEV)
    y, _ = wqp.rms_norm(x, w, 1e-6)
    assert y[0].isfinite().all() and not y[1].any() and y[4].isfinite().all()
    assert y[2, 3].isnan() and not y[2, :3].any() and y[3].isnan().all()
    c, s, _ = wqp.rms_norm_a8(x, w, 1e-6)
    assert s[2, 0].isnan() and s[3].isnan().all() and s[0].isfinite().all() and not e4m3(c)[1].any()
    assert wqp.rms_norm(x[1:2], w, 0.0)[0].isnan().all()           # 0 * (1 / 0)


# ---------------------------------------------------------------- products
def w4_operand(R, K, seed, ints):
    g = gen(seed)
    codes = torch.randint(0, 256, (R, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    if ints:      # values 0, +-1, +-2 with scales 1 and 2: sums are integers below 2^24 for K <= 2^18
        nib = torch.tensor([0, 2, 4, 10, 12], dtype=torch.uint8, device=DEV)[torch.randint(0, 5, (R, K), generator=g, device=DEV)]
        codes = nib[:, 0::2] | (nib[:, 1::2] << 4)
        scales = torch.tensor([0x38, 0x40], dtype=torch.uint8, device=DEV)[torch.randint(0, 2, (R, K // 16), generator=g, device=DEV)]
    else:
        scales = (torch.rand((R, K // 16), generator=g, device=DEV) * 3).to(torch.float8_e4m3fn).view(torch.uint8)
    v = E2M1.to(DEV)[torch.stack((codes & 15, codes >> 4), 2).view(R, K).long()]
    v = (v.view(R, -1, 16) * scales.view(torch.float8_e4m3fn).double().unsqueeze(2)).view(R, K)
    return codes, scales, v


def w8_operand(R, K, seed, ints, block):
    g = gen(seed)
    if ints:
        q = torch.randint(-3, 4, (R, K), generator=g, device=DEV).float()
    else:
        q = torch.randn((R, K), generator=g, device=DEV) * 20
    codes = q.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    shape = ((R + 127) // 128, K // 128) if block else (R, K // 128)
    scales = torch.rand(shape, generator=g, device=DEV) * 2
    if ints:
        scales = torch.where(scales > 1, 2.0, 1.0)
    s = scales.double().repeat_interleave(128, 1)
    s = s.repeat_interleave(128, 0)[:R] if block else s
    return codes, scales.contiguous(), codes.view(torch.float8_e4m3fn).double() * s


def run(fmt, M, N, K, seed, ints, out=None, g=(1.0, 1.0)):
    if fmt == 4:
        a, sa, av = w4_operand(M, K, seed, ints)
        w, sw, wv = w4_operand(N, K, seed + 1, ints)
        C = wqp.w4a4_gemm(a, sa, w, sw, N, K, g[0], g[1], out=out)
    else:
        a, sa, av = w8_operand(M, K, seed, ints, False)
        w, sw, wv = w8_operand(N, K, seed + 1, ints, True)
        C = wqp.w8a8_gemm(a, sa, w, sw, N, K, out=out)
    return C, av, wv


def check(C, av, wv, K, ints, g=1.0):
    ref = (av @ wv.t()) * g
    if ints:
        assert torch.equal(C, ref.float().bfloat16())
        return
    tol = 2.0 ** -8 * ref.abs() + (K / 32 + 16) * 2.0 ** -22 * (av.abs() @ wv.abs().t()) * g
    assert ((C.double() - ref).abs() <= tol).all()


# Every tile width and kernel of both: few rows with K split 1 to 4 ways, many rows, edges in M and N.
SHAPES = [(1, 1, 256), (1, 128, 512), (2, 129, 2560), (7, 5000, 768), (16, 127, 1024), (17, 300, 1280), (32, 1000, 256),
          (33, 257, 2048), (64, 640, 5120), (65, 130, 1024), (96, 2000, 512), (128, 384, 1536), (129, 255, 256), (200, 64, 768),
          (256, 256, 512), (257, 1, 1024), (300, 5001, 512), (511, 193, 256), (600, 3000, 256), (1025, 700, 768), (130, 20000, 256),
          (40, 20000, 512), (5, 20000, 256)]


@pytest.mark.parametrize("fmt", [4, 8])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_products(fmt, M, N, K):
    for ints in (True, False):
        C, av, wv = run(fmt, M, N, K, seed=M + N + K, ints=ints)
        check(C, av, wv, K, ints)
    assert wqp.get_device_error() == 0


@pytest.mark.parametrize("fmt,K", [(4, 65536), (8, 65536), (8, 128), (8, 16512), (4, 17408)])
@pytest.mark.parametrize("M", [1, 50, 300])
def test_products_long_and_short_k(fmt, K, M):
    C, av, wv = run(fmt, M, 260, K, seed=K + M, ints=True)
    check(C, av, wv, K, True)


@pytest.mark.parametrize("fmt", [4, 8])
@pytest.mark.parametrize("M,N,K", [(3, 2, 15616), (20, 1100, 5120), (53, 5, 16896), (65, 300, 10240), (129, 100, 5120), (257, 145, 11264),
                                   (300, 640, 10240), (1000, 256, 5120), (1146, 21, 14336), (1985, 39, 12800), (17, 19999, 768),
                                   (32, 20000, 2560), (49, 19510, 768), (64, 34816, 1280), (100, 20002, 768), (128, 34816, 2560),
                                   (384, 34817, 512)])
def test_products_with_k_split_and_with_many_tiles(fmt, M, N, K):
    """Few tiles with a long K, with one and with many rows per tile, and more tiles than SMs, into rows that are 13
    elements longer."""
    buf = torch.full((M + 2, N + 13), 7.0, dtype=torch.bfloat16, device=DEV).view(-1)
    out = torch.as_strided(buf, (M, N), (N + 13, 1), N + 14)
    for ints in (True, False):
        C, av, wv = run(fmt, M, N, K, seed=M + N, ints=ints, out=out)
        check(C, av, wv, K, ints)
    out.fill_(7.0)
    assert (buf == 7.0).all()
    assert wqp.get_device_error() == 0


# A pair of CTAs takes two or three tiles of 128, 256 and 192 columns, with fewer 128-K blocks a tile than it has accumulators.
@pytest.mark.parametrize("M,N", [(7680, 640), (9728, 1024), (2560, 2048), (7681, 2050)])
@pytest.mark.parametrize("K", [128, 256, 384])
def test_w8a8_tiles_shorter_than_the_accumulators(M, N, K):
    C, av, wv = run(8, M, N, K, seed=M + K, ints=True)
    check(C, av, wv, K, True)
    assert wqp.get_device_error() == 0


@pytest.mark.parametrize("fmt", [4, 8])
@pytest.mark.parametrize("M,N,pad,shift", [(3, 131, 5, 0), (40, 256, 8, 8), (300, 256, 8, 0), (300, 260, 4, 0), (300, 256, 1, 0),
                                           (300, 256, 8, 1), (300, 256, 8, 3), (270, 131, 13, 0)])
def test_products_into_pitched_rows(fmt, M, N, pad, shift):
    """Rows of C that are and are not 16-byte aligned; what lies between and around them stays."""
    K = 512
    buf = torch.full((M + 2, N + pad), 7.0, dtype=torch.bfloat16, device=DEV).view(-1)
    out = torch.as_strided(buf, (M, N), (N + pad, 1), N + pad + shift)
    C, av, wv = run(fmt, M, N, K, seed=N + pad, ints=True, out=out)
    assert C is out
    check(C, av, wv, K, True)
    out.fill_(7.0)
    assert (buf == 7.0).all()


@pytest.mark.parametrize("M", [1, 33, 300])
def test_w4a4_global_scales(M):
    C, av, wv = run(4, M, 200, 768, seed=M, ints=False, g=(0.0625, 3.0))
    check(C, av, wv, 768, False, g=0.0625 * 3.0)


@pytest.mark.parametrize("M", [2, 300])
def test_w4a4_negative_and_nan_scales(M):
    """A scale code is a magnitude: one with its sign bit set, like the NaN code, makes its row's outputs NaN."""
    N, K = 140, 512
    a, sa, av = w4_operand(M, K, 1, True)
    w, sw, wv = w4_operand(N, K, 2, True)
    a |= 0x22                                   # no zero codes: every product meets its scale
    sw[5, 3], sw[137, 31], sa[1, 17] = 0xB8, 0x7F, 0x80
    C = wqp.w4a4_gemm(a, sa, w, sw, N, K)
    bad = torch.zeros((M, N), dtype=torch.bool, device=DEV)
    bad[:, 5], bad[:, 137], bad[1, :] = True, True, True
    assert torch.equal(C.isnan(), bad)


def test_w8a8_nan_reaches_its_row_only():
    M, N, K = 40, 200, 256
    a, sa, _ = w8_operand(M, K, 1, True, False)
    w, sw, _ = w8_operand(N, K, 2, True, True)
    a[3, 130] = 0x7F
    sa[9, 1] = float("nan")
    C = wqp.w8a8_gemm(a, sa, w, sw, N, K)
    assert C[3].isnan().all() and C[9].isnan().all() and int(C.isnan().sum()) == 2 * N


@pytest.mark.parametrize("fmt", [4, 8])
def test_products_over_many_rows_in_pieces(fmt):
    """More than 2^20 rows: C's offsets pass 2^31 bytes, and the last piece is one row."""
    M, N, K = (1 << 20) + 1, 1040, 256
    C, av, wv = run(fmt, M, N, K, seed=3, ints=True)
    for at in (slice(0, 300), slice((1 << 20) - 150, M)):
        check(C[at], av[at], wv, K, True)


@pytest.mark.parametrize("fmt,M", [(4, 1), (4, 300), (8, 20), (8, 300)])
def test_products_repeat_bit_for_bit(fmt, M):
    first = run(fmt, M, 1000, 2560, seed=8, ints=False)[0]
    for _ in range(4):
        assert torch.equal(run(fmt, M, 1000, 2560, seed=8, ints=False)[0], first)


# ---------------------------------------------------------------- together
def layer(x, r, w, w8, s8, w4, s4, stream=None):
    """norm -> 8-bit product -> 4-bit quantisation -> 4-bit product, on one stream."""
    K, N = x.shape[1], w8.shape[0]
    c, s, h = wqp.rms_norm_a8(x, w, 1e-6, residual=r, stream=stream)
    u = wqp.w8a8_gemm(c, s, w8, s8, N, K, stream=stream)
    q, qs = wqp.w4_quantize(u, 0.5, stream=stream)
    return wqp.w4a4_gemm(q, qs, w4, s4, K, N, 0.5, 1.0, stream=stream), h, u


@pytest.mark.parametrize("M", [1, 24, 200, 700])
def test_chain_under_pdl_and_on_a_side_stream(M):
    K, N = 5120, 1024
    x, r = rows(M, K, torch.bfloat16, 0, 1), rows(M, K, torch.bfloat16, 0, 2)
    w = torch.ones(K, dtype=torch.bfloat16, device=DEV)
    w8, s8, _ = w8_operand(N, K, 3, False, True)
    w4, s4, _ = w4_operand(K, N, 4, False)
    want = layer(x, r, w, w8, s8, w4, s4)
    assert want[0].isfinite().all()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = layer(x, r, w, w8, s8, w4, s4, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    old = wqp.set_pdl(True)
    try:
        for _ in range(5):
            got = layer(x, r, w, w8, s8, w4, s4)
            assert all(torch.equal(a, b) for a, b in zip(want, got))
    finally:
        wqp.set_pdl(old)
    assert wqp.get_device_error() == 0


@pytest.mark.parametrize("M", [3, 200])
def test_chain_in_a_cuda_graph(M):
    """Captured once, replayed on new inputs in the same buffers."""
    K, N = 1024, 512
    x, r = rows(M, K, torch.bfloat16, 0, 1), rows(M, K, torch.bfloat16, 0, 2)
    w = torch.ones(K, dtype=torch.bfloat16, device=DEV)
    w8, s8, _ = w8_operand(N, K, 3, False, True)
    w4, s4, _ = w4_operand(K, N, 4, False)
    layer(x, r, w, w8, s8, w4, s4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(x, r, w, w8, s8, w4, s4)
    for seed in (11, 12):
        x.copy_(rows(M, K, torch.bfloat16, 0, seed))
        graph.replay()
        want = layer(x, r, w, w8, s8, w4, s4)
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_binding_refuses():
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(256, dtype=torch.bfloat16, device=DEV)
    c, s = wqp.w4_quantize(x)
    c8, s8 = wqp.a8_quantize(x)
    f = s8.new_zeros(1, 2)
    bad = [
        (TypeError, lambda: wqp.w4_quantize(x.double())), (ValueError, lambda: wqp.w4_quantize(x.t())),
        (ValueError, lambda: wqp.w4_quantize(x[0])), (ValueError, lambda: wqp.w4_quantize(x, 1.0, out=(c, s[:2]))),
        (TypeError, lambda: wqp.a8_quantize(x, out=(c8, c8))), (wqp.WqpError, lambda: wqp.a8_quantize(x[:, :200])),
        (wqp.WqpError, lambda: wqp.w4_quantize(x, 0.0)), (wqp.WqpError, lambda: wqp.w4_quantize(x[:, 4:132])),
        (ValueError, lambda: wqp.rms_norm(x, w[:128], 1e-6)), (ValueError, lambda: wqp.rms_norm(x, w.float(), 1e-6)),
        (ValueError, lambda: wqp.rms_norm(x, w, 1e-6, residual=x[:2])), (ValueError, lambda: wqp.rms_norm(x, w, 1e-6, residual_out=x)),
        (ValueError, lambda: wqp.rms_norm(x, w, 1e-6, residual=x, residual_out=x.float())), (wqp.WqpError, lambda: wqp.rms_norm(x, w, -1.0)),
        (ValueError, lambda: wqp.w4a4_gemm(c, s, c, s, 5, 256)), (ValueError, lambda: wqp.w4a4_gemm(c, s[:, :8], c, s, 4, 256)),
        (TypeError, lambda: wqp.w4a4_gemm(c.int(), s, c, s, 4, 256)), (TypeError, lambda: wqp.w4a4_gemm(c, s, c, s, 4, 256, out=x.float()[:, :4])),
        (ValueError, lambda: wqp.w4a4_gemm(c, s, c, s, 4, 256, out=x)), (TypeError, lambda: wqp.w8a8_gemm(c8, s8, c8, f.half(), 4, 256)),
        (ValueError, lambda: wqp.w8a8_gemm(c8, s8, c8, s8, 4, 256)), (ValueError, lambda: wqp.w8a8_gemm(c8[:, ::2], s8, c8, f, 4, 256)),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()
    assert wqp.w4a4_gemm(c[:0], s[:0], c, s, 4, 256).shape == (0, 4)
    assert wqp.rms_norm(x[:0], w, 1e-6)[0].shape == (0, 256) and wqp.w4_quantize(x[:0])[0].shape == (0, 128)


@pytest.mark.parametrize("pitch", [5, 5 * 2 ** 30, 2 ** 32 + 2048])
def test_a_single_row_of_any_stride(pitch):
    """[1, T, K][:, -1] has one row, T * K elements from the next: the stride means nothing."""
    N, K = 256, 1024
    x, r = rows(1, K, torch.bfloat16, 0, 1), rows(1, K, torch.bfloat16, 0, 2)
    w = torch.ones(K, dtype=torch.bfloat16, device=DEV)
    w8, s8, _ = w8_operand(N, K, 3, True, True)
    one = lambda t: torch.as_strided(t, t.shape, (pitch, 1))
    assert all(torch.equal(a, b) for a, b in zip(wqp.w4_quantize(x), wqp.w4_quantize(one(x))))
    assert all(torch.equal(a, b) for a, b in zip(wqp.rms_norm(x, w, 1e-6, residual=r),
                                                 wqp.rms_norm(one(x), w, 1e-6, residual=one(r), residual_out=one(r.clone()), out=one(x.clone()))))
    out = torch.empty(1, N, dtype=torch.bfloat16, device=DEV)
    want = wqp.w8a16_gemm(x, w8, s8, N, K)
    assert torch.equal(wqp.w8a16_gemm(one(x), w8, s8, N, K, out=one(out)), want) and torch.equal(out, want)


def test_example_runs():
    """The example's block with quantised activations is near the one without: E2M1 rows and weights keep about
    three significant bits, so their product over many K is a few percent to a tenth off."""
    import examples.quantised_ffn as ex

    found = ex.main(["--hidden", "512", "--ffn", "1024", "--rows", "1,200"])
    assert [f[0] for f in found] == [1, 200] and all(f[1] < 0.25 for f in found)
