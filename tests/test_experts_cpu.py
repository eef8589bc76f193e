"""Refusals of the experts' entries: every bad argument is turned away by the C ABI before any CUDA call, and by the
binding before the ABI."""
from __future__ import annotations

import ctypes

import pytest
import torch

P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(8)]
OFF8, OFF2, OFF1 = ctypes.c_void_p(0x10008), ctypes.c_void_p(0x10002), ctypes.c_void_p(0x10001)
NUL = ctypes.c_void_p(0)
INVALID = 1
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    from weight_only_quantized_packed_gb300 import build

    build.build()
    from weight_only_quantized_packed_gb300 import binding

    return binding.lib()


# (position, bad value, a word of the reason) against a call that is right otherwise.
#        logits ldl dtype bias ids weights T E k scoring groups top_groups best renorm scale
ROUTE = [P[0], 64, 2, P[1], P[2], P[3], 5, 64, 6, 1, 8, 3, 2, 1, 1.0, NUL]
ORDER = [P[0], P[1], P[2], 40, 16, NUL]
#          A lda W scales globals rows offsets C ldc T slots E N K gated workspace
EXPERTS = [P[0], 256, P[1], P[2], P[3], P[4], P[5], P[6], 40, 3, 2, 8, 40, 256, 0, P[7], NUL]
#          Y ldy weights ids E residual ldr out ldo dtype T slots H
COMBINE = [P[0], 256, P[1], P[2], 8, P[3], 256, P[4], 256, 0, 3, 2, 256, NUL]

CASES = (
    [("expert_route", ROUTE, *c) for c in [
        (0, NUL, "NULL"), (0, OFF2, "aligned"), (1, 63, "pitch"), (2, 3, "dtype"), (2, -1, "dtype"), (3, OFF2, "bias"), (4, NUL, "ids"),
        (4, OFF2, "ids"), (5, NUL, "weights"), (5, OFF1, "weights"), (6, -1, "T="), (6, 1 << 29, "pairs"), (7, 0, "E="), (7, 1025, "E="),
        (7, 60, "groups="), (8, 0, "slots"), (8, 33, "slots"), (8, 25, "top_k="), (9, 2, "scoring"), (9, -1, "scoring"), (10, 0, "groups="),
        (10, 64, "groups="), (10, 7, "groups="), (11, 0, "top_groups="), (11, 9, "top_groups="), (12, 0, "group_best"), (12, 3, "group_best"),
        (14, NAN, "scale"), (14, INF, "scale")]]
    + [("expert_order", ORDER, *c) for c in [
        (0, NUL, "ids"), (0, OFF2, "ids"), (1, NUL, "rows"), (1, OFF1, "rows"), (2, NUL, "offsets"), (2, OFF2, "offsets"), (3, -1, "R="),
        (3, (1 << 30) + 1, "R="), (4, 0, "E="), (4, 1025, "E=")]]
    + [("w4a16_experts", EXPERTS, *c) for c in [
        (0, NUL, "NULL A"), (0, OFF8, "16-byte"), (1, 248, "pitch"), (1, 260, "pitch"), (2, NUL, "NULL"), (2, OFF8, "16-byte"), (3, NUL, "NULL"),
        (3, OFF8, "16-byte"), (4, OFF2, "global_scales"), (5, NUL, "rows"), (5, OFF2, "rows"), (6, NUL, "offsets"), (6, OFF1, "offsets"),
        (7, NUL, "NULL"), (7, OFF1, "2-byte"), (8, 39, "ldc"), (9, -1, "T="), (9, 1 << 30, "pairs"), (10, 0, "slots"), (10, 33, "slots"),
        (11, 0, "E="), (11, 1025, "E="), (12, 0, "N="), (12, (1 << 24) + 1, "N="), (13, 0, "K="), (13, 192, "K="), (13, (1 << 20) + 128, "K="), (15, OFF8, "workspace")]]
    + [("expert_combine", COMBINE, *c) for c in [
        (0, NUL, "NULL Y"), (0, OFF8, "16-byte"), (1, 248, "pitch"), (1, 260, "pitch"), (2, NUL, "weights"), (2, OFF2, "weights"), (3, NUL, "ids"),
        (3, OFF2, "ids"), (4, 0, "E="), (4, 1025, "E="), (5, OFF8, "residual"), (6, 128, "residual"), (7, NUL, "out"), (7, OFF8, "out"),
        (8, 248, "out"), (9, 3, "dtype"), (10, -1, "T="), (11, 0, "slots"), (11, 33, "slots"), (12, 252, "H="), (12, 0, "H="),
        (12, (1 << 20) + 8, "H=")]]
)


@pytest.mark.parametrize("name,good,at,bad,word", CASES)
def test_abi_refuses(L, name, good, at, bad, word):
    args = list(good)
    args[at] = bad
    assert getattr(L, name)(*args) == INVALID, (name, args)
    said = L.wqp_last_error().decode()
    assert said.startswith(name) and word in said, said


def test_abi_refuses_an_odd_gated_n(L):
    args = list(EXPERTS)
    args[12], args[14] = 39, 1
    assert L.w4a16_experts(*args) == INVALID and "even" in L.wqp_last_error().decode()


@pytest.mark.parametrize("name,args,t", [("expert_route", ROUTE, 6), ("w4a16_experts", EXPERTS, 9), ("expert_combine", COMBINE, 10)])
def test_no_tokens_is_a_no_op(L, name, args, t):
    args = [NUL if isinstance(a, ctypes.c_void_p) else a for a in args]
    args[t] = 0
    assert getattr(L, name)(*args) == 0


def test_binding_refuses_host_tensors(L):
    import weight_only_quantized_packed_gb300 as wqp

    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    w, s = torch.zeros(4, 8, 128, dtype=torch.uint8), torch.zeros(4, 8, 16, dtype=torch.uint8)
    ids, weights = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1)
    rows, offsets = torch.zeros(2, dtype=torch.int32), torch.zeros(5, dtype=torch.int32)
    for call in (lambda: wqp.expert_route(x, 2), lambda: wqp.expert_order(ids, 4),
                 lambda: wqp.w4a16_experts(x, w, s, rows, offsets, 8, 256), lambda: wqp.expert_combine(x, weights, ids, 4)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
