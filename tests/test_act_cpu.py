"""Refusals of the quantised-activation entries: every bad argument is turned
away by the C ABI before any CUDA call, and by the binding before the ABI."""
from __future__ import annotations

import ctypes

import pytest
import torch

P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(6)]
OFF8, OFF2, OFF1 = ctypes.c_void_p(0x10008), ctypes.c_void_p(0x10002), ctypes.c_void_p(0x10001)
NUL = ctypes.c_void_p(0)
INVALID = 1


@pytest.fixture(scope="module")
def L():
    from weight_only_quantized_packed_gb300 import build

    build.build()
    from weight_only_quantized_packed_gb300 import binding

    return binding.lib()


def refused(L, name, args, word):
    assert getattr(L, name)(*args) == INVALID, (name, args)
    said = L.wqp_last_error().decode()
    assert said.startswith(name) and word in said, said


# (position, bad value, a word of the reason) against a call that is right otherwise.
W4Q = [P[0], 256, 0, 1.0, P[1], P[2], 4, 256, NUL]
A8Q = [P[0], 256, 0, P[1], P[2], 4, 256, NUL]
NORM = [P[0], 256, P[1], 256, P[2], 1e-6, P[3], 256, P[4], 256, 0, 4, 256, NUL]
NORM8 = [P[0], 256, P[1], 256, P[2], 1e-6, P[3], 256, P[4], P[5], 0, 4, 256, NUL]
GEMM4 = [P[0], P[1], 1.0, P[2], P[3], 1.0, P[4], 40, 4, 40, 512, NUL]
GEMM8 = [P[0], P[1], P[2], P[3], P[4], 40, 4, 40, 384, NUL]
NAN = float("nan")

CASES = (
    [("w4_quantize", W4Q, *c) for c in [
        (0, NUL, "NULL X"), (0, OFF8, "16-byte"), (1, 248, "pitch"), (1, 260, "pitch"), (2, 3, "dtype"), (2, -1, "dtype"),
        (3, NAN, "global_scale"), (3, 0.0, "global_scale"), (3, -1.0, "global_scale"), (3, float("inf"), "global_scale"),
        (4, NUL, "NULL"), (4, OFF2, "8-byte"), (5, NUL, "NULL"), (6, -1, "M="), (7, 200, "K="), (7, 0, "K="),
        (7, (1 << 20) + 128, "K=")]]
    + [("a8_quantize", A8Q, *c) for c in [
        (0, NUL, "NULL X"), (0, OFF8, "16-byte"), (1, 128, "pitch"), (2, 7, "dtype"), (3, OFF2, "8-byte"), (4, OFF2, "4-byte"),
        (5, -2, "M="), (6, 130, "K=")]]
    + [("rms_norm", NORM, *c) for c in [
        (0, NUL, "NULL X"), (1, 255, "pitch"), (2, OFF8, "residual"), (3, 252, "residual"), (4, NUL, "weight"), (4, OFF8, "weight"),
        (5, NAN, "eps"), (5, -1e-9, "eps"), (5, float("inf"), "eps"), (6, OFF8, "residual_out"), (7, 128, "residual_out"),
        (8, NUL, "NULL Y"), (8, OFF8, "Y"), (9, 8, "Y"), (10, 3, "dtype"), (11, -1, "M="), (12, 64, "K=")]]
    + [("rms_norm_a8", NORM8, *c) for c in [
        (0, OFF8, "X"), (8, NUL, "NULL codes"), (8, OFF2, "8-byte"), (9, OFF2, "4-byte"), (5, NAN, "eps"), (12, 100, "K=")]]
    + [("w4a4_gemm", GEMM4, *c) for c in [
        (0, NUL, "NULL"), (0, OFF8, "16-byte"), (1, OFF8, "16-byte"), (2, NAN, "NaN"), (3, OFF8, "16-byte"), (4, NUL, "NULL"),
        (5, NAN, "NaN"), (6, NUL, "NULL"), (6, OFF1, "2-byte"), (7, 39, "ldc"), (8, -1, "M="), (9, 0, "N="),
        (9, (1 << 24) + 1, "N="), (10, 384, "K="), (10, 0, "K="), (10, (1 << 20) + 256, "K=")]]
    + [("w8a8_gemm", GEMM8, *c) for c in [
        (0, OFF8, "16-byte"), (1, OFF2, "4-byte"), (2, NUL, "NULL"), (3, OFF2, "4-byte"), (4, OFF1, "2-byte"), (5, 12, "ldc"),
        (6, -3, "M="), (7, -1, "N="), (8, 200, "K=")]]
)


@pytest.mark.parametrize("name,good,at,bad,word", CASES)
def test_abi_refuses(L, name, good, at, bad, word):
    args = list(good)
    args[at] = bad
    refused(L, name, args, word)


@pytest.mark.parametrize("name,args,m", [("w4_quantize", W4Q, 6), ("a8_quantize", A8Q, 5), ("rms_norm", NORM, 11),
                                         ("rms_norm_a8", NORM8, 11), ("w4a4_gemm", GEMM4, 8), ("w8a8_gemm", GEMM8, 6)])
def test_no_rows_is_a_no_op(L, name, args, m):
    """M = 0 returns OK without looking at the pointers (an empty tensor has none)."""
    args = [NUL if isinstance(a, ctypes.c_void_p) else a for a in args]
    args[m] = 0
    assert getattr(L, name)(*args) == 0


def test_binding_refuses_host_tensors(L):
    import weight_only_quantized_packed_gb300 as wqp

    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    c4, s4 = torch.zeros(2, 128, dtype=torch.uint8), torch.zeros(2, 16, dtype=torch.uint8)
    c8, s8 = torch.zeros(2, 256, dtype=torch.uint8), torch.zeros(2, 2)
    for call in (lambda: wqp.w4_quantize(x), lambda: wqp.a8_quantize(x), lambda: wqp.rms_norm(x, x[0], 1e-6),
                 lambda: wqp.rms_norm_a8(x, x[0], 1e-6), lambda: wqp.w4a4_gemm(c4, s4, c4, s4, 2, 256),
                 lambda: wqp.w8a8_gemm(c8, s8, c8, s8, 2, 256)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
