"""What the binding does around a call, without a GPU: stand-ins for the library, for device tensors and for torch's
allocator record which arguments arrive and from which stream's pool an output comes."""
from __future__ import annotations

import contextlib
import types

import pytest
import torch

from weight_only_quantized_packed_gb300 import binding

CURRENT, SIDE = 0x1000, 0x2000


class Tensor:
    """Looks like a device tensor to the binding."""

    is_cuda = True
    device = "cuda:0"

    def __init__(self, shape, dtype, strides=None, pool=None):
        self.shape, self.dtype, self.pool, self.recorded = torch.Size(shape), dtype, pool, []
        if strides is None:
            strides = [1] * len(self.shape)
            for i in range(len(self.shape) - 2, -1, -1):
                strides[i] = strides[i + 1] * self.shape[i + 1]
        self.strides = tuple(strides)

    def stride(self, i=None):
        return self.strides if i is None else self.strides[i]

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return all(s == t for s, t in zip(self.strides, Tensor(self.shape, None).strides))

    def data_ptr(self):
        return 0x10000

    def record_stream(self, stream):
        self.recorded.append(stream.cuda_stream)


class Stream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle


class Library:
    """Every entry returns OK and is noted with its arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def world(monkeypatch):
    """The stand-ins in the binding's place: .calls of the library, .made by the allocator."""
    state = types.SimpleNamespace(stream=Stream(CURRENT), made=[])

    @contextlib.contextmanager
    def on(stream):
        old, state.stream = state.stream, stream
        yield
        state.stream = old

    def empty(*shape, dtype, device):
        t = Tensor(shape[0] if len(shape) == 1 else shape, dtype, pool=state.stream.cuda_stream)
        state.made.append(t)
        return t

    cuda = types.SimpleNamespace(stream=on, Stream=Stream, ExternalStream=Stream, current_stream=lambda *_: state.stream,
                                 default_stream=lambda *_: Stream(0))
    fake = types.SimpleNamespace(empty=empty, cuda=cuda, uint8=torch.uint8, bfloat16=torch.bfloat16, float16=torch.float16,
                                 float32=torch.float32)
    binding._load_torch()                           # fills the dtype table from the real one
    monkeypatch.setattr(binding, "_torch", fake)
    monkeypatch.setattr(binding, "_lib", Library())
    monkeypatch.setattr(binding, "_current_stream", lambda: state.stream.cuda_stream)
    state.calls = binding._lib.calls
    return state


def bf16(*shape, strides=None):
    return Tensor(shape, torch.bfloat16, strides)


def u8(*shape):
    return Tensor(shape, torch.uint8)


def f32(*shape):
    return Tensor(shape, torch.float32)


M, N, K = 3, 640, 1024
# Every entry that makes its outputs: a call of it, and how many it makes.
MAKERS = {
    "w4_quantize": (lambda **k: binding.w4_quantize(bf16(M, K), 1.0, **k), 2),
    "a8_quantize": (lambda **k: binding.a8_quantize(bf16(M, K), **k), 2),
    "rms_norm": (lambda **k: binding.rms_norm(bf16(M, K), bf16(K), 1e-6, residual=bf16(M, K), **k), 2),
    "rms_norm_a8": (lambda **k: binding.rms_norm_a8(bf16(M, K), bf16(K), 1e-6, residual=bf16(M, K), **k), 3),
    "w4a4_gemm": (lambda **k: binding.w4a4_gemm(u8(M, K // 2), u8(M, K // 16), u8(N, K // 2), u8(N, K // 16), N, K, **k), 1),
    "w8a8_gemm": (lambda **k: binding.w8a8_gemm(u8(M, K), f32(M, K // 128), u8(N, K), f32(N // 128, K // 128), N, K, **k), 1),
    **{n: (lambda n=n, **k: getattr(binding, n)(bf16(M, K), u8(N, K * 34 // 128), N, K, **k), 1)
       for n in ("q2_gemv", "q2_gemm_tc", "q2_gemm_mma")},
    **{n: (lambda n=n, **k: getattr(binding, n)(bf16(M, K), u8(N, K), u8(N, K // 16), N, K, **k), 1)
       for n in ("w4a16_gemv", "w4a16_gemm_tc", "w4a16_gemm_mma", "w8a16_gemm", "w8a16_gemm_tc", "w8a16_gemm_mma")},
    "q2_dequant": (lambda **k: binding.q2_dequant(u8(N, K * 34 // 128), N, K, **k), 1),
    "w4a16_dequant": (lambda **k: binding.w4a16_dequant(u8(N, K // 2), u8(N, K // 16), N, K, **k), 1),
    "w8a16_dequant": (lambda **k: binding.w8a16_dequant(u8(N, K), f32(N // 128, K // 128), N, K, **k), 1),
}


@pytest.mark.parametrize("name", sorted(MAKERS))
@pytest.mark.parametrize("given", [Stream(SIDE), SIDE, 0], ids=["stream", "handle", "default"])
def test_outputs_come_from_the_stream_that_is_passed(world, name, given):
    """A block of the current stream's pool may still be in use there, and goes back there while the passed stream
    uses it. The current stream, which may read the output later, is recorded."""
    call, count = MAKERS[name]
    call(stream=given)
    handle = given.cuda_stream if isinstance(given, Stream) else given
    assert [t.pool for t in world.made] == [handle] * count
    assert [t.recorded for t in world.made] == [[CURRENT]] * count
    assert world.calls[-1][1][-1] == handle


@pytest.mark.parametrize("name", sorted(MAKERS))
@pytest.mark.parametrize("given", [None, Stream(CURRENT), CURRENT], ids=["none", "stream", "handle"])
def test_outputs_on_the_current_stream_are_plain(world, name, given):
    call, count = MAKERS[name]
    call(stream=given)
    assert [(t.pool, t.recorded) for t in world.made] == [(CURRENT, [])] * count
    assert world.calls[-1][1][-1] == CURRENT


# Pitches: (entry, call with rows of the given strides, position of the pitch in the library's arguments, pitch of contiguous rows).
def _gemm4(C):
    return binding.w4a4_gemm(u8(2, K // 2), u8(2, K // 16), u8(N, K // 2), u8(N, K // 16), N, K, out=C)


def _gemm8(C):
    return binding.w8a8_gemm(u8(2, K), f32(2, K // 128), u8(N, K), f32(N // 128, K // 128), N, K, out=C)


def _norm(x=None, r=None, h=None, y=None, m=2):
    return binding.rms_norm(x or bf16(m, K), bf16(K), 1e-6, residual=r or bf16(m, K), residual_out=h, out=y)


def _norm8(x=None, r=None, h=None, m=2):
    return binding.rms_norm_a8(x or bf16(m, K), bf16(K), 1e-6, residual=r or bf16(m, K), residual_out=h)


PITCHED = [
    ("w4_quantize x", K, 1, lambda t: binding.w4_quantize(t, 1.0)), ("a8_quantize x", K, 1, binding.a8_quantize),
    ("rms_norm x", K, 1, lambda t: _norm(x=t, m=t.shape[0])), ("rms_norm residual", K, 3, lambda t: _norm(r=t, m=t.shape[0])),
    ("rms_norm residual_out", K, 7, lambda t: _norm(h=t, m=t.shape[0])), ("rms_norm out", K, 9, lambda t: _norm(y=t, m=t.shape[0])),
    ("rms_norm_a8 x", K, 1, lambda t: _norm8(x=t, m=t.shape[0])), ("rms_norm_a8 residual", K, 3, lambda t: _norm8(r=t, m=t.shape[0])),
    ("rms_norm_a8 residual_out", K, 7, lambda t: _norm8(h=t, m=t.shape[0])),
]
for _n, _w in [("q2_gemv", (u8(N, K * 34 // 128),)), ("q2_gemm_tc", (u8(N, K * 34 // 128),)), ("q2_gemm_mma", (u8(N, K * 34 // 128),))] + [
        (n, (u8(N, K), u8(N, K // 16)))
        for n in ("w4a16_gemv", "w4a16_gemm_tc", "w4a16_gemm_mma", "w8a16_gemm", "w8a16_gemm_tc", "w8a16_gemm_mma")]:
    PITCHED += [(_n + " A", K, 1, lambda t, n=_n, w=_w: getattr(binding, n)(t, *w, N, K)),
                (_n + " out", N, {1: 4, 2: 5}[len(_w)] + _n.startswith("w4"),
                 lambda t, n=_n, w=_w: getattr(binding, n)(bf16(t.shape[0], K), *w, N, K, out=t))]
PITCHED_OUT = [("w4a4_gemm out", N, 7, _gemm4), ("w8a8_gemm out", N, 5, _gemm8)]


@pytest.mark.parametrize("pitch", [2 ** 31, 2 ** 32 + 2048, 5 * 2 ** 30])
@pytest.mark.parametrize("name,cols,at,call", PITCHED + PITCHED_OUT, ids=[p[0] for p in PITCHED + PITCHED_OUT])
def test_pitches_beyond_an_int_are_refused(world, name, cols, at, call, pitch):
    """The C ABI takes a pitch as an int: a larger one would arrive as another pitch."""
    with pytest.raises(ValueError, match="pitch"):
        call(bf16(2, cols, strides=(pitch, 1)))
    assert not world.calls


@pytest.mark.parametrize("name,cols,at,call", PITCHED + PITCHED_OUT, ids=[p[0] for p in PITCHED + PITCHED_OUT])
def test_the_largest_pitch_arrives(world, name, cols, at, call):
    call(bf16(2, cols, strides=(2 ** 31 - 8, 1)))
    assert world.calls[-1][1][at] == 2 ** 31 - 8


@pytest.mark.parametrize("pitch", [5, 5 * 2 ** 30, 2 ** 32 + 2048])
@pytest.mark.parametrize("name,cols,at,call", PITCHED, ids=[p[0] for p in PITCHED])
def test_one_row_has_no_pitch(world, name, cols, at, call, pitch):
    """The last token of one long sequence: [1, T, K][:, -1] is T * K apart from nothing."""
    call(bf16(1, cols, strides=(pitch, 1)))
    assert world.calls[-1][1][at] == cols
