"""Rows of very small activations, BF16's subnormal numbers among them, in the entries that scale activations to FP16.

A BF16 number below 2^-126 is a multiple of 2^-133. Scaled by at most 2^109 all of them are FP16 numbers, so where a row's
magnitudes lie below 2^-95 nothing of it is rounded, and the tolerances are those of ordinary rows: tests/test_gpu_experts.py's
(which allows for rounded activations besides) and the scalar term. Global and block scales bring the outputs into BF16's
normal range. A single product of 8-bit and 6-bit significands is an FP32 number, and the output is its rounding to BF16,
bit for bit; times 2^100 or 2^60, a power of two, too.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import weight_only_quantized_packed_gb300 as wqp
from tests import _gpu as G
from tests._tol import assert_scalar_term
from tests.test_gpu_experts import DEV, experts64, gen, make_experts
from weight_only_quantized_packed_gb300 import synth

pytestmark = pytest.mark.gpu
EXPONENTS = [-86, -95, -96, -100, -108, -112, -116, -120, -126, -131]


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert wqp.get_device_error() == 0


@pytest.mark.parametrize("e", EXPONENTS)
@pytest.mark.parametrize("T", [2, 60])                       # few pairs an expert, many
@pytest.mark.parametrize("gated", [False, True])
def test_experts(e, T, gated):
    E, k, N, K = 2, 2, 48, 640
    g = gen(15 - e)
    w, s, gs = make_experts(E, N, K, 16)
    a = (torch.randn((T, K), generator=g, device=DEV).double() * 2.0 ** e).bfloat16()
    a[0, 1:] = 0                                             # a row of one element
    a[1] = 0
    gs = gs * 2.0 ** 100
    ids = torch.randint(0, E, (T, k), generator=g, device=DEV, dtype=torch.int32)
    got = wqp.w4a16_experts(a, w, s, *wqp.expert_order(ids, E), N, K, gs, gated).double().cpu()
    want, tol, _ = experts64(a, w, s, gs, ids, gated, k)
    assert ((got - want).abs() <= tol).all(), float(((got - want).abs() / tol).max())
    assert (got[2:2 * k] == 0).all()


@pytest.mark.parametrize("pairs", ["few", "many"])
def test_experts_every_exponent_alone(pairs):
    """Rows of one element with all significant bits set, for every exponent from BF16's subnormals to 2^-80."""
    bits = torch.cat((torch.tensor([1, 3, 7, 15, 31, 63, 127]), torch.arange(1, 48) * 128 + 127)).to(torch.int16)
    T, E, N, K = len(bits), 60 if pairs == "few" else 3, 20, 256
    a = torch.zeros((T, K), dtype=torch.int16)
    at = (torch.arange(T) * 37) % K
    a[torch.arange(T), at] = bits
    a = a.view(torch.bfloat16).to(DEV)
    w, s, _ = make_experts(E, N, K, 17)
    ids = (torch.arange(T, dtype=torch.int32) % E).view(T, 1).to(DEV)
    gs = torch.full((E,), 2.0 ** 100, device=DEV)
    got = wqp.w4a16_experts(a, w, s, *wqp.expert_order(ids, E), N, K, gs)
    want, _, _ = experts64(a, w, s, gs, ids, False, 1)
    assert (want != 0).any(1).all() and torch.equal(got.cpu().float(), want.float().bfloat16().float())


@pytest.mark.parametrize("fmt", ["w4", "w8"])
@pytest.mark.parametrize("N", [300, 20001])                  # for W4A16: one short CTA a tile, the persistent kernel
@pytest.mark.parametrize("e", EXPONENTS)
def test_mma_entries(oracle_lib, fmt, N, e):
    M, K = 9, 2048
    d = G.make(fmt, M, N, K, seed=83)
    A = synth.bf16_bits_from_f32((synth.bf16_bits_to_f32(d["A"]).astype(np.float64) * 2.0 ** e).astype(np.float32))
    # The oracle sums products in FP32, where those of small rows are subnormal: it gets the rows times 2^64, which is exact,
    # and the scales times 2^-64.
    up = synth.bf16_bits_from_f32(synth.bf16_bits_to_f32(A) * np.float32(2.0 ** 64))
    d.update(A=up, dA=G.dev_bf16(A))
    if fmt == "w4":
        ref = G.run_oracle(oracle_lib, dict(d, g=1.37 * 2.0 ** -4))
        d["g"] = 1.37 * 2.0 ** 60
    else:
        ref = G.run_oracle(oracle_lib, dict(d, S=d["S"] * np.float32(2.0 ** -4)))
        d["dS"] = G.dev_f32(d["S"] * np.float32(2.0 ** 60))
    assert_scalar_term(G.host_bits(G.run_gpu(d, tc="mma")), ref, K, f"{fmt} mma N={N} activations of 2^{e}")


@pytest.mark.parametrize("e,scale", [(-86, -30), (-100, -20), (-100, -30), (-108, -20), (-60, -60), (100, -60), (100, 10)])
def test_w8_mma_with_small_and_large_block_scales(oracle_lib, e, scale):
    """Outputs in BF16's range whose two scales' product FP32 does not hold, or barely."""
    M, N, K = 4, 300, 2048
    d = G.make("w8", M, N, K, seed=84)
    A = synth.bf16_bits_from_f32((synth.bf16_bits_to_f32(d["A"]).astype(np.float64) * 2.0 ** e).astype(np.float32))
    r = np.random.default_rng(85)
    S = ((1.0 + r.random(d["S"].shape)) * 2.0 ** scale).astype(np.float32)
    W = synth.e4m3_round(r.integers(-448, 449, size=(N, K)).astype(np.float64))
    d.update(A=A, dA=G.dev_bf16(A), S=S, dS=G.dev_f32(S), W=W, dW=G.dev_u8(W))
    assert_scalar_term(G.host_bits(G.run_gpu(d, tc="mma")), G.run_oracle(oracle_lib, d), K, f"w8 mma 2^{e}, scales 2^{scale}")
