"""Refusals of the experts' entries: every bad argument is turned away by the C ABI before any CUDA call, and by the
binding before the ABI."""
from __future__ import annotations

import ctypes

import pytest
import torch

from tests.test_binding_cpu import CURRENT, SIDE, Stream, Tensor, world  # noqa: F401 (world is a fixture)

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


# ---------------------------------------------------------------- the binding, with stand-ins
class Here(Tensor):
    """A stand-in of the device `place`."""

    place = 0

    def get_device(self):
        return self.place


def t(dtype, *shape, strides=None, place=0):
    x = Here(shape, dtype, strides)
    x.place = place
    return x


def bf16(*shape, **k):
    return t(torch.bfloat16, *shape, **k)


def f32(*shape, **k):
    return t(torch.float32, *shape, **k)


def i32(*shape, **k):
    return t(torch.int32, *shape, **k)


def u8(*shape, **k):
    return t(torch.uint8, *shape, **k)


@pytest.fixture
def experts(world, monkeypatch):  # noqa: F811
    from weight_only_quantized_packed_gb300 import binding

    binding._torch.int32 = torch.int32
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    made, empty = world.made, binding._torch.empty

    def here(*shape, dtype, device):
        out = empty(*shape, dtype=dtype, device=device)
        out.get_device = lambda: 0
        return out

    binding._torch.empty = here
    world.need = 0
    binding._lib.w4a16_experts_workspace = lambda *a: world.need
    return world


T, k, E, N, K, H = 6, 2, 4, 48, 256, 128


def call(name, **kw):
    from weight_only_quantized_packed_gb300 import binding as b

    return {
        "expert_route": lambda: b.expert_route(kw.pop("x", f32(T, E)), k, **kw),
        "expert_order": lambda: b.expert_order(kw.pop("x", i32(T, k)), E, **kw),
        "w4a16_experts": lambda: b.w4a16_experts(kw.pop("x", bf16(T, K)), kw.pop("w", u8(E, N, K // 2)), u8(E, N, K // 16), kw.pop("rows", i32(T * k)),
                                                 i32(E + 1), N, K, **kw),
        "expert_combine": lambda: b.expert_combine(kw.pop("x", bf16(T * k, H)), f32(T, k), kw.pop("ids", i32(T, k)), E, **kw),
    }[name]()


MAKES = {"expert_route": 2, "expert_order": 2, "w4a16_experts": 1, "expert_combine": 1}


@pytest.mark.parametrize("name", sorted(MAKES))
@pytest.mark.parametrize("need", [0, 4096])
def test_outputs_and_workspace_come_from_the_stream_that_is_passed(experts, name, need):
    experts.need = need
    call(name, stream=Stream(SIDE))
    count = MAKES[name] + (1 if need and name == "w4a16_experts" else 0)
    assert [m.pool for m in experts.made] == [SIDE] * count and [m.recorded for m in experts.made] == [[CURRENT]] * count
    assert experts.calls[-1][0] == name and experts.calls[-1][1][-1] == SIDE
    experts.made.clear()
    call(name)
    assert [(m.pool, m.recorded) for m in experts.made] == [(CURRENT, [])] * count


@pytest.mark.parametrize("name", sorted(MAKES))
def test_another_device_is_refused(experts, name):
    x = {"expert_route": f32(T, E, place=1), "expert_order": i32(T, k, place=1), "w4a16_experts": bf16(T, K, place=1),
         "expert_combine": bf16(T * k, H, place=1)}[name]
    with pytest.raises(ValueError, match="current device"):
        call(name, x=x)
    assert not experts.calls


def test_binding_refuses_what_does_not_fit(experts):
    for name, kw, kind, word in [
            ("expert_route", {"scoring": "relu"}, ValueError, "scoring"), ("expert_route", {"bias": f32(E + 1)}, ValueError, "bias"),
            ("expert_route", {"bias": bf16(E)}, TypeError, "bias"), ("expert_route", {"x": i32(T, E)}, TypeError, "logits"),
            ("expert_route", {"out": (i32(T, k + 1), f32(T, k))}, ValueError, "ids"), ("expert_route", {"out": (i32(T, k), bf16(T, k))}, TypeError, "weights"),
            ("expert_order", {"x": t(torch.int64, T, k)}, TypeError, "ids"), ("expert_order", {"x": i32(T, k, strides=(1, T))}, ValueError, "ids"),
            ("expert_order", {"out": (i32(T * k), i32(E))}, ValueError, "offsets"),
            ("w4a16_experts", {"x": bf16(5, K)}, ValueError, "pairs"), ("w4a16_experts", {"x": f32(T, K)}, TypeError, "A"),
            ("w4a16_experts", {"w": u8(E, N, K)}, ValueError, "W"), ("w4a16_experts", {"global_scales": f32(E - 1)}, ValueError, "global_scales"),
            ("w4a16_experts", {"gated": True, "out": bf16(T * k, N)}, ValueError, "out"), ("w4a16_experts", {"rows": bf16(T * k)}, TypeError, "rows"),
            ("expert_combine", {"x": bf16(T * k + 1, H)}, ValueError, "weights"), ("expert_combine", {"ids": i32(T * k)}, ValueError, "ids"),
            ("expert_combine", {"residual": f32(T, H)}, ValueError, "residual"), ("expert_combine", {"out": bf16(T * k, H)}, ValueError, "out"),
            ("w4a16_experts", {"x": bf16(T, K, strides=(2 ** 31, 1))}, ValueError, "pitch"),
            ("w4a16_experts", {"out": bf16(T * k, N, strides=(2 ** 31, 1))}, ValueError, "pitch"),
            ("expert_combine", {"x": bf16(T * k, H, strides=(2 ** 31, 1))}, ValueError, "pitch"),
            ("expert_combine", {"out": bf16(T, H, strides=(2 ** 31, 1))}, ValueError, "pitch"),
            ("expert_route", {"x": f32(T, E, strides=(2 ** 31, 1))}, ValueError, "pitch")]:
        with pytest.raises(kind, match=word):
            call(name, **kw)
    assert not experts.calls


def test_arguments_arrive(experts):
    call("w4a16_experts", x=bf16(T * k, K, strides=(K + 8, 1)), gated=True)       # a row of its own for each pair
    assert experts.calls[-1][1][1] == K + 8 and experts.calls[-1][1][8:15] == (N // 2, T * k, 1, E, N, K, 1)
    call("w4a16_experts")
    assert experts.calls[-1][1][8:15] == (N, T, k, E, N, K, 0) and experts.calls[-1][1][15] is None
    res = bf16(T, H, strides=(H + 8, 1))
    call("expert_combine", residual=res, out=res)
    assert experts.calls[-1][1][1] == H and experts.calls[-1][1][6] == experts.calls[-1][1][8] == H + 8
    call("expert_route", x=f32(T, E, strides=(E + 3, 1)), scoring="sigmoid", renormalise=False, scale=2.5)
    assert experts.calls[-1][1][1:3] == (E + 3, 2) and experts.calls[-1][1][6:15] == (T, E, k, 1, 1, 1, 2, 0, 2.5)


def test_workspace_sizes(L):
    """Small calls need none; where it is needed, a row of K halves and a factor for each pair."""
    size = L.w4a16_experts_workspace
    assert size(1, 8, 128, 4096, 5120) == 0 and size(0, 1, 8, 64, 256) == 0
    assert size(4096, 8, 128, 4096, 5120) == 32768 * (5120 * 2 + 4)
    assert size(1 << 20, 8, 8, 64, 4096) == (8 << 20) * (4096 * 2 + 4)            # beyond 32 bits
    for bad in [(-1, 8, 8, 64, 256), (4, 33, 8, 64, 256), (4, 2, 0, 64, 256), (4, 2, 8, 0, 256), (4, 2, 8, 64, 200)]:
        assert size(*bad) == 0
    args = list(EXPERTS)
    args[9], args[10], args[15] = 100, 8, NUL
    assert size(100, 8, 8, 40, 256) and L.w4a16_experts(*args) == INVALID and "workspace" in L.wqp_last_error().decode()


BIG = [2 ** 31, 2 ** 32 + 2, -2 ** 32 + 2]


@pytest.mark.parametrize("big", BIG)
def test_sizes_beyond_an_int_are_refused(experts, big):
    """The C ABI takes sizes as ints: a larger one would arrive as another size, and the call succeed for that one."""
    from weight_only_quantized_packed_gb300 import binding as b

    if big > 0:
        for what, run in [
                ("T=", lambda: b.expert_route(f32(big, 2), 1)), ("R=", lambda: b.expert_order(i32(big, 1), E)),
                ("slots=", lambda: b.w4a16_experts(bf16(1, K), u8(E, N, K // 2), u8(E, N, K // 16), i32(big), i32(E + 1), N, K)),
                ("E=", lambda: b.w4a16_experts(bf16(T, K), u8(big, N, K // 2), u8(big, N, K // 16), i32(T * k), i32(big + 1), N, K)),
                ("T=", lambda: b.expert_combine(bf16(big, 8), f32(big, 1), i32(big, 1), E)),
                ("slots=", lambda: b.expert_combine(bf16(big, 8), f32(1, big), i32(1, big), E))]:
            with pytest.raises(ValueError, match=what):
                run()
    for name, kw in [("expert_route", {"groups": big}), ("expert_route", {"top_groups": big}), ("expert_route", {"group_best": big})]:
        with pytest.raises(ValueError, match=next(iter(kw))):
            call(name, **kw)
    for what, run in [("top_k=", lambda: b.expert_route(f32(T, E), big)), ("E=", lambda: b.expert_order(i32(T, k), big)),
                      ("E=", lambda: b.expert_combine(bf16(T * k, H), f32(T, k), i32(T, k), big))]:
        with pytest.raises(ValueError, match=what):
            run()
    assert not experts.calls and not experts.made
