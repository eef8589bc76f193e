"""Thin ctypes binding over libwqp.so (the C ABI declared in include/wqp.h).

Argument marshalling only. torch supplies device memory and the current
stream, and every step of the computation runs in the library's CUDA
kernels. There is no CPU or PyTorch fallback: if libwqp.so is missing or a
call fails, an exception is raised.

Every call takes ``stream`` (a stream object or a handle; the current stream
without one). Outputs it makes belong to that stream, as if made under
``torch.cuda.stream(stream)``, and may be read on the stream that is current
after that one has been waited for. Operands are the caller's: complete before
the call runs, and kept (or given to ``Tensor.record_stream``) until it has.
"""
from __future__ import annotations

import ctypes
import os
import threading

__all__ = [
    "WqpError", "lib", "lib_path", "q2_gemv", "q2_gemm_tc", "q2_gemm_mma", "w4a16_gemv", "w4a16_gemm_tc",
    "w4a16_gemm_mma", "w8a16_gemm", "w8a16_gemm_tc", "w8a16_gemm_mma",
    "w4_quantize", "a8_quantize", "rms_norm", "rms_norm_a8", "w4a4_gemm", "w8a8_gemm",
    "expert_route", "expert_order", "w4a16_experts", "expert_combine",
    "q2_dequant", "w4a16_dequant", "w8a16_dequant", "row_chunks", "set_pdl",
    "get_device_error", "selftest_wait_timeout", "status_string", "EXPORTS", "MAX_M_PER_LAUNCH",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libwqp.so")
MAX_M_PER_LAUNCH = 16

_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float

# name -> argtypes; every symbol declared in include/wqp.h.
EXPORTS = {
    "q2_gemv": [_P, _P, _P, _P, _I, _I, _I, _P],
    "q2_gemv_strided": [_P, _I, _P, _P, _I, _I, _I, _I, _P],
    "q2_gemm_tc": [_P, _P, _P, _I, _I, _I, _P],
    "q2_gemm_tc_strided": [_P, _I, _P, _P, _I, _I, _I, _I, _P],
    "q2_gemm_mma": [_P, _P, _P, _I, _I, _I, _P],
    "q2_gemm_mma_strided": [_P, _I, _P, _P, _I, _I, _I, _I, _P],
    "w4a16_gemv": [_P, _P, _P, _P, _I, _I, _I, _P],
    "w4a16_gemv_ex": [_P, _I, _P, _P, _F, _P, _I, _I, _I, _I, _P],
    "w4a16_gemm_tc": [_P, _P, _P, _P, _I, _I, _I, _P],
    "w4a16_gemm_tc_ex": [_P, _I, _P, _P, _F, _P, _I, _I, _I, _I, _P],
    "w4a16_gemm_mma": [_P, _P, _P, _P, _I, _I, _I, _P],
    "w4a16_gemm_mma_ex": [_P, _I, _P, _P, _F, _P, _I, _I, _I, _I, _P],
    "w8a16_gemm": [_P, _P, _P, _P, _I, _I, _I, _P],
    "w8a16_gemm_strided": [_P, _I, _P, _P, _P, _I, _I, _I, _I, _P],
    "w8a16_gemm_tc": [_P, _P, _P, _P, _I, _I, _I, _P],
    "w8a16_gemm_tc_strided": [_P, _I, _P, _P, _P, _I, _I, _I, _I, _P],
    "w8a16_gemm_mma": [_P, _P, _P, _P, _I, _I, _I, _P],
    "w8a16_gemm_mma_strided": [_P, _I, _P, _P, _P, _I, _I, _I, _I, _P],
    "w4_quantize": [_P, _I, _I, _F, _P, _P, _I, _I, _P],
    "a8_quantize": [_P, _I, _I, _P, _P, _I, _I, _P],
    "rms_norm": [_P, _I, _P, _I, _P, _F, _P, _I, _P, _I, _I, _I, _I, _P],
    "rms_norm_a8": [_P, _I, _P, _I, _P, _F, _P, _I, _P, _P, _I, _I, _I, _P],
    "w4a4_gemm": [_P, _P, _F, _P, _P, _F, _P, _I, _I, _I, _I, _P],
    "w8a8_gemm": [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P],
    "expert_route": [_P, _I, _I, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P],
    "expert_order": [_P, _P, _P, _I, _I, _P],
    "w4a16_experts": [_P, _I, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P],
    "w4a16_experts_workspace": [_I, _I, _I, _I, _I],
    "expert_combine": [_P, _I, _P, _P, _I, _P, _I, _P, _I, _I, _I, _I, _I, _P],
    "q2_dequant": [_P, _P, _I, _I, _P],
    "w4a16_dequant": [_P, _P, _F, _P, _I, _I, _P],
    "w8a16_dequant": [_P, _P, _P, _I, _I, _P],
    "wqp_row_chunks": [_I, _I, _I, _I, ctypes.POINTER(ctypes.c_longlong), _I],
    "wqp_set_pdl": [_I],
    "wqp_get_device_error": [],
    "wqp_selftest_wait_timeout": [_I, _P],
    "wqp_status_string": [_I],
    "wqp_last_error": [],
    "wqp_abi_version": [],
}

_lock = threading.Lock()
_lib = None


class WqpError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}" + (f" ({detail})" if detail else ""))


def lib() -> ctypes.CDLL:
    """Load libwqp.so (built in-tree by ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(lib_path):
                raise ImportError(
                    f"libwqp.so not found at {lib_path}; build it with "
                    "`python -c 'import __graft_entry__ as g; g.build()'`")
            L = ctypes.CDLL(lib_path)
            for name, args in EXPORTS.items():
                fn = getattr(L, name)
                fn.argtypes = args
                fn.restype = _I
            L.wqp_status_string.restype = ctypes.c_char_p
            L.wqp_last_error.restype = ctypes.c_char_p
            L.w4a16_experts_workspace.restype = ctypes.c_size_t
            _lib = L
    return _lib


def status_string(status: int) -> str:
    try:
        return lib().wqp_status_string(int(status)).decode()
    except ImportError:
        return f"status {status}"


def _check(status: int, where: str):
    if status != 0:
        raise WqpError(status, where, lib().wqp_last_error().decode())


_current_stream = None   # () -> raw handle of this thread's current stream, set on first use
_BF16 = None


def _stream(stream):
    """The stream argument as an integer handle (ctypes converts it)."""
    global _current_stream
    if stream is None:
        if _current_stream is None:
            import torch

            # The current stream's raw handle; torch.cuda.current_stream()
            # builds a Python stream object, which costs about as much host
            # time as a launch.
            raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
            if raw is not None:
                dev = torch._C._cuda_getDevice
                _current_stream = lambda: raw(dev())
            else:
                _current_stream = lambda: torch.cuda.current_stream().cuda_stream
        return _current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t):
    """A tensor's device address as an integer (None for no tensor)."""
    return t.data_ptr() if t is not None else None


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors (no CPU fallback)")


def _empty(shape, dtype, device, stream):
    """A new output for a call on `stream` (its argument, not the handle)."""
    torch = _torch
    if stream is None or _stream(stream) == _stream(None):
        return torch.empty(shape, dtype=dtype, device=device)
    # From the pool of the call's stream: a block of the current stream's may
    # still be in use by work queued there. The current stream is recorded, so
    # that the block is not handed out again while it is read there.
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)
        stream = torch.cuda.ExternalStream(handle, device) if handle > 1 else torch.cuda.default_stream(device)
    current = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        out = torch.empty(shape, dtype=dtype, device=device)
    out.record_stream(current)
    return out


def _out(A, M, N, out, stream):
    if out is None:
        out = _empty((M, N), (_torch or _load_torch()).bfloat16, A.device, stream)
    return out


_INT_MAX = 2 ** 31 - 1


def _too_far(name, ld):
    raise ValueError(f"{name}: a row pitch of {ld} elements is more than 2^31 - 1")


def _pitch(name, t):
    """The row pitch of [M, K] as the C ABI takes it, in an int: ctypes would cut a larger one without a word. A
    single row has none, whatever its stride."""
    shape = t.shape
    ld = t.stride(0) if shape[0] > 1 else shape[1]
    if ld > _INT_MAX:
        _too_far(name, ld)
    return ld


def _rows(A, K):
    global _BF16
    if _BF16 is None:
        import torch

        _BF16 = torch.bfloat16
    if A.dtype is not _BF16:
        raise TypeError("A must be torch.bfloat16")
    if A.dim() != 2 or A.shape[1] != K or A.stride(1) != 1:
        raise ValueError(f"A must be [M, {K}] with unit column stride")
    return A.shape[0], _pitch("A", A)


def q2_gemv(A, W, N: int, K: int, out=None, stream=None):
    """C[M, N] = A @ dequant_q2(W)^T. W is uint8 Q2_0 blocks (34*K/128 B per row)."""
    _need_cuda(A, W, out)
    M, lda = _rows(A, K)
    C = _out(A, M, N, out, stream)
    _check(lib().q2_gemv_strided(_ptr(A), lda, _ptr(W), _ptr(C), _pitch("out", C), M, N, K,
                                 _stream(stream)), "q2_gemv")
    return C


def q2_gemm_tc(A, W, N: int, K: int, out=None, stream=None):
    """Tensor-core (tcgen05 swap-AB) form of q2_gemv, 1 <= M <= 16, K % 1024 == 0."""
    _need_cuda(A, W, out)
    M, lda = _rows(A, K)
    C = _out(A, M, N, out, stream)
    _check(lib().q2_gemm_tc_strided(_ptr(A), lda, _ptr(W), _ptr(C), _pitch("out", C), M, N, K,
                                    _stream(stream)), "q2_gemm_tc")
    return C


def q2_gemm_mma(A, W, N: int, K: int, out=None, stream=None):
    """Warp-level tensor-core (mma.sync swap-AB) form of q2_gemv, 1 <= M <= 16, K % 1024 == 0."""
    _need_cuda(A, W, out)
    M, lda = _rows(A, K)
    C = _out(A, M, N, out, stream)
    _check(lib().q2_gemm_mma_strided(_ptr(A), lda, _ptr(W), _ptr(C), _pitch("out", C), M, N, K,
                                     _stream(stream)), "q2_gemm_mma")
    return C


def w4a16_gemv(A, W, scales, N: int, K: int, global_scale: float = 1.0, out=None, stream=None):
    """C = A @ dequant_w4(W, scales, global_scale)^T."""
    _need_cuda(A, W, scales, out)
    M, lda = _rows(A, K)
    C = _out(A, M, N, out, stream)
    _check(lib().w4a16_gemv_ex(_ptr(A), lda, _ptr(W), _ptr(scales), float(global_scale), _ptr(C),
                               _pitch("out", C), M, N, K, _stream(stream)), "w4a16_gemv")
    return C


def w4a16_gemm_tc(A, W, scales, N: int, K: int, global_scale: float = 1.0, out=None, stream=None):
    """Tensor-core (tcgen05 swap-AB) form of w4a16_gemv, 1 <= M <= 16, K % 256 == 0."""
    _need_cuda(A, W, scales, out)
    M, lda = _rows(A, K)
    C = _out(A, M, N, out, stream)
    _check(lib().w4a16_gemm_tc_ex(_ptr(A), lda, _ptr(W), _ptr(scales), float(global_scale), _ptr(C),
                                  _pitch("out", C), M, N, K, _stream(stream)), "w4a16_gemm_tc")
    return C


def w4a16_gemm_mma(A, W, scales, N: int, K: int, global_scale: float = 1.0, out=None, stream=None):
    """Warp-level tensor-core (mma.sync swap-AB) form of w4a16_gemv, K % 1024 == 0."""
    _need_cuda(A, W, scales, out)
    M, lda = _rows(A, K)
    C = _out(A, M, N, out, stream)
    _check(lib().w4a16_gemm_mma_ex(_ptr(A), lda, _ptr(W), _ptr(scales), float(global_scale), _ptr(C),
                                   _pitch("out", C), M, N, K, _stream(stream)), "w4a16_gemm_mma")
    return C


def w8a16_gemm_mma(A, W, scales, N: int, K: int, out=None, stream=None):
    """Warp-level tensor-core (mma.sync swap-AB) form of w8a16_gemm, K % 1024 == 0."""
    _need_cuda(A, W, scales, out)
    M, lda = _rows(A, K)
    C = _out(A, M, N, out, stream)
    _check(lib().w8a16_gemm_mma_strided(_ptr(A), lda, _ptr(W), _ptr(scales), _ptr(C), _pitch("out", C),
                                        M, N, K, _stream(stream)), "w8a16_gemm_mma")
    return C


def w8a16_gemm(A, W, scales, N: int, K: int, out=None, stream=None):
    """C = A @ (e4m3(W) * block_scales)^T, scalar-FMA kernels."""
    _need_cuda(A, W, scales, out)
    M, lda = _rows(A, K)
    C = _out(A, M, N, out, stream)
    _check(lib().w8a16_gemm_strided(_ptr(A), lda, _ptr(W), _ptr(scales), _ptr(C), _pitch("out", C),
                                    M, N, K, _stream(stream)), "w8a16_gemm")
    return C


def w8a16_gemm_tc(A, W, scales, N: int, K: int, out=None, stream=None):
    """Tensor-core (tcgen05 swap-AB) form of w8a16_gemm, 1 <= M <= 16."""
    _need_cuda(A, W, scales, out)
    M, lda = _rows(A, K)
    C = _out(A, M, N, out, stream)
    _check(lib().w8a16_gemm_tc_strided(_ptr(A), lda, _ptr(W), _ptr(scales), _ptr(C), _pitch("out", C),
                                       M, N, K, _stream(stream)), "w8a16_gemm_tc")
    return C


_DTYPES = {}             # torch dtype -> wqp_dtype, filled on first use
_torch = None


def _load_torch():
    """torch, once: an import statement on every call costs a tenth of a launch."""
    global _torch
    if _torch is None:
        import torch

        _DTYPES.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2})
        _torch = torch
    return _torch


# _typed_rows, _rows_like and _gemm_out have _pitch's lines in place of a call,
# which costs a twentieth of a small call's host time (w4_quantize 4.9 -> 5.2 us).
def _typed_rows(name, x):
    """Rows [M, K] with unit column stride: (pitch, wqp_dtype, M, K)."""
    if not x.is_cuda:
        raise ValueError("all tensors must be CUDA tensors (no CPU fallback)")
    dt = _DTYPES.get(x.dtype)
    if dt is None:
        raise TypeError(f"{name} must be torch.bfloat16, float16 or float32")
    shape, stride = x.shape, x.stride()
    if len(shape) != 2 or (stride[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name} must be [M, K] with unit column stride")
    M, K = shape
    ld = stride[0] if M > 1 else K
    if ld > _INT_MAX:
        _too_far(name, ld)
    return ld, dt, M, K


def _rows_like(name, t, x):
    """The pitch of rows with the shape and type of x."""
    if not t.is_cuda:
        raise ValueError("all tensors must be CUDA tensors (no CPU fallback)")
    shape, stride = t.shape, t.stride()
    if t.dtype is not x.dtype or shape != x.shape or (stride[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name} must have the shape and type of x, with unit column stride")
    ld = stride[0] if shape[0] > 1 else shape[1]
    if ld > _INT_MAX:
        _too_far(name, ld)
    return ld


def _packed(name, t, shape, dtype):
    """A contiguous tensor of a packed format; its address."""
    if not t.is_cuda:
        raise ValueError("all tensors must be CUDA tensors (no CPU fallback)")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {list(shape)} tensor")
    return t.data_ptr()


def _weights(name, t, count, dtype):
    """Packed weights or their scales (any shape, as the GEMV entries take them); their address."""
    if not t.is_cuda:
        raise ValueError("all tensors must be CUDA tensors (no CPU fallback)")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.numel() != count or not t.is_contiguous():
        raise ValueError(f"{name} must hold {count} contiguous values")
    return t.data_ptr()


def _codes_out(x, codes_shape, scales_shape, scales_dtype, out, stream):
    """(codes, scales), new or the caller's."""
    if out is None:
        return (_empty(codes_shape, _torch.uint8, x.device, stream),
                _empty(scales_shape, scales_dtype, x.device, stream))
    codes, scales = out
    if not (codes.is_cuda and scales.is_cuda):
        raise ValueError("all tensors must be CUDA tensors (no CPU fallback)")
    if codes.dtype is not _torch.uint8 or scales.dtype is not scales_dtype:
        raise TypeError(f"out must be torch.uint8 codes and {scales_dtype} scales")
    if (codes.shape != codes_shape or scales.shape != scales_shape
            or not (codes.is_contiguous() and scales.is_contiguous())):
        raise ValueError(f"out must be contiguous {list(codes_shape)} codes and {list(scales_shape)} scales")
    return codes, scales


def w4_quantize(x, global_scale: float = 1.0, out=None, stream=None):
    """Rows x [M, K] (bfloat16, float16 or float32) to the W4A16 format: uint8 codes [M, K/2] and
    uint8 E4M3 scales [M, K/16], under one global_scale. out: (codes, scales) to write to."""
    torch = _torch or _load_torch()
    ldx, dt, M, K = _typed_rows("x", x)
    codes, scales = _codes_out(x, (M, K // 2), (M, K // 16), torch.uint8, out, stream)
    status = (_lib or lib()).w4_quantize(x.data_ptr(), ldx, dt, float(global_scale), codes.data_ptr(),
                                         scales.data_ptr(), M, K, _stream(stream))
    if status:
        _check(status, "w4_quantize")
    return codes, scales


def a8_quantize(x, out=None, stream=None):
    """Rows x [M, K] (bfloat16, float16 or float32) to uint8 E4M3 codes [M, K] with float32 scales
    [M, K/128]. out: (codes, scales) to write to."""
    torch = _torch or _load_torch()
    ldx, dt, M, K = _typed_rows("x", x)
    codes, scales = _codes_out(x, (M, K), (M, K // 128), torch.float32, out, stream)
    status = (_lib or lib()).a8_quantize(x.data_ptr(), ldx, dt, codes.data_ptr(), scales.data_ptr(), M, K,
                                         _stream(stream))
    if status:
        _check(status, "a8_quantize")
    return codes, scales


def _norm_args(x, weight, residual, residual_out, stream):
    """(residual's address and pitch, residual_out, its address and pitch, weight's address)."""
    K = x.shape[1]
    if not weight.is_cuda:
        raise ValueError("all tensors must be CUDA tensors (no CPU fallback)")
    if weight.dtype is not x.dtype or weight.shape != (K,) or not weight.is_contiguous():
        raise ValueError(f"weight must be a contiguous [{K}] tensor of x's type")
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out without residual")
        return None, 0, None, None, 0, weight.data_ptr()
    ldr = _rows_like("residual", residual, x)
    if residual_out is None:
        residual_out, ldh = _empty(x.shape, x.dtype, x.device, stream), K
    else:
        ldh = ldr if residual_out is residual else _rows_like("residual_out", residual_out, x)
    return residual.data_ptr(), ldr, residual_out, residual_out.data_ptr(), ldh, weight.data_ptr()


def rms_norm(x, weight, eps: float, residual=None, residual_out=None, out=None, stream=None):
    """(y, h): h = x + residual, y = h * rsqrt(mean(h^2) + eps) * weight, in x's type (bfloat16,
    float16 or float32). Without a residual h is None. residual_out may be the residual itself."""
    torch = _torch or _load_torch()
    ldx, dt, M, K = _typed_rows("x", x)
    pr, ldr, h, ph, ldh, pw = _norm_args(x, weight, residual, residual_out, stream)
    if out is None:
        out, ldy = _empty((M, K), x.dtype, x.device, stream), K
    else:
        ldy = _rows_like("out", out, x)
    status = (_lib or lib()).rms_norm(x.data_ptr(), ldx, pr, ldr, pw, float(eps), ph, ldh, out.data_ptr(), ldy,
                                      dt, M, K,
                                      _stream(stream))
    if status:
        _check(status, "rms_norm")
    return out, h


def rms_norm_a8(x, weight, eps: float, residual=None, residual_out=None, out=None, stream=None):
    """(codes, scales, h): rms_norm with y written as a8_quantize writes it. out: (codes, scales)."""
    torch = _torch or _load_torch()
    ldx, dt, M, K = _typed_rows("x", x)
    pr, ldr, h, ph, ldh, pw = _norm_args(x, weight, residual, residual_out, stream)
    codes, scales = _codes_out(x, (M, K), (M, K // 128), torch.float32, out, stream)
    status = (_lib or lib()).rms_norm_a8(x.data_ptr(), ldx, pr, ldr, pw, float(eps), ph, ldh, codes.data_ptr(),
                                         scales.data_ptr(), dt, M, K,
                                         _stream(stream))
    if status:
        _check(status, "rms_norm_a8")
    return codes, scales, h


def _gemm_out(A, M, N, out, stream):
    if out is None:
        return _empty((M, N), _torch.bfloat16, A.device, stream), N
    if not out.is_cuda:
        raise ValueError("all tensors must be CUDA tensors (no CPU fallback)")
    if out.dtype is not _torch.bfloat16:
        raise TypeError("out must be torch.bfloat16")
    stride = out.stride()
    if out.shape != (M, N) or (stride[1] != 1 and N > 1):
        raise ValueError(f"out must be [{M}, {N}] with unit column stride")
    ldc = stride[0] if M > 1 else N
    if ldc > _INT_MAX:
        _too_far("out", ldc)
    return out, ldc


def w4a4_gemm(A, a_scales, W, w_scales, N: int, K: int, a_global: float = 1.0, w_global: float = 1.0, out=None,
              stream=None):
    """C[M, N] = dequant(A) @ dequant(W)^T, both in the W4A16 format (w4_quantize), any M, K % 256 == 0."""
    torch = _torch or _load_torch()
    M, u8 = A.shape[0], torch.uint8
    pa, psa = _packed("A", A, (M, K // 2), u8), _packed("a_scales", a_scales, (M, K // 16), u8)
    pw, psw = _weights("W", W, N * (K // 2), u8), _weights("w_scales", w_scales, N * (K // 16), u8)
    C, ldc = _gemm_out(A, M, N, out, stream)
    status = (_lib or lib()).w4a4_gemm(pa, psa, float(a_global), pw, psw, float(w_global), C.data_ptr(), ldc, M, N, K,
                                       _stream(stream))
    if status:
        _check(status, "w4a4_gemm")
    return C


def w8a8_gemm(A, a_scales, W, w_scales, N: int, K: int, out=None, stream=None):
    """C[M, N] = dequant(A) @ dequant(W)^T: A as a8_quantize and rms_norm_a8 write it, W8A16 weights, any M."""
    torch = _torch or _load_torch()
    M = A.shape[0]
    pa, psa = _packed("A", A, (M, K), torch.uint8), _packed("a_scales", a_scales, (M, K // 128), torch.float32)
    pw = _weights("W", W, N * K, torch.uint8)
    psw = _weights("w_scales", w_scales, (N + 127) // 128 * (K // 128), torch.float32)
    C, ldc = _gemm_out(A, M, N, out, stream)
    status = (_lib or lib()).w8a8_gemm(pa, psa, pw, psw, C.data_ptr(), ldc, M, N, K, _stream(stream))
    if status:
        _check(status, "w8a8_gemm")
    return C


_SCORING = {"softmax": 0, "sigmoid": 1}
_current_device = None   # () -> index of this thread's current device, set on first use


def _here(*ts):
    """The experts' entries take tensors of the current device: the library launches there."""
    global _current_device
    if _current_device is None:
        _load_torch()
        _current_device = getattr(_torch._C, "_cuda_getDevice", None) or _torch.cuda.current_device
    device = -1
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors (no CPU fallback)")
        if device < 0:
            device = _current_device()
        if t.get_device() != device:
            raise ValueError("all tensors must be on the current device")


def _ints(names, *values):
    """Sizes and counts go to the C ABI as ints: ctypes would cut others without a word."""
    if max(values) > _INT_MAX or min(values) < -_INT_MAX:
        bad = [f"{n}={v}" for n, v in zip(names.split(), values) if abs(v) > _INT_MAX]
        raise ValueError(f"{', '.join(bad)}: beyond 2^31 - 1")


def expert_route(logits, top_k: int, scoring: str = "softmax", bias=None, groups: int = 1, top_groups: int = 1,
                 group_best: int = 2, renormalise: bool = True, scale: float = 1.0, out=None, stream=None):
    """(ids, weights): each token's top_k experts from its logits [T, E] (bfloat16, float16 or float32) by score
    ("softmax" or "sigmoid") plus bias (float32 [E]), of the top_groups best of `groups` groups of experts; int32 ids and
    float32 weights [T, top_k], the scores, renormalised to sum to 1 and times scale. Id -1: no expert was left (logits
    of -inf). out: (ids, weights) to write to."""
    torch = _torch or _load_torch()
    _here(logits, bias)
    ldl, dt, T, E = _typed_rows("logits", logits)
    _ints("T E top_k groups top_groups group_best", T, E, top_k, groups, top_groups, group_best)
    if scoring not in _SCORING:
        raise ValueError("scoring must be 'softmax' or 'sigmoid'")
    pb = None if bias is None else _packed("bias", bias, (E,), torch.float32)
    if out is None:
        ids, weights = (_empty((T, top_k), torch.int32, logits.device, stream),
                        _empty((T, top_k), torch.float32, logits.device, stream))
    else:
        ids, weights = out
        _here(ids, weights)
        _packed("ids", ids, (T, top_k), torch.int32)
        _packed("weights", weights, (T, top_k), torch.float32)
    status = (_lib or lib()).expert_route(logits.data_ptr(), ldl, dt, pb, ids.data_ptr(), weights.data_ptr(), T, E, top_k,
                                          _SCORING[scoring], groups, top_groups, group_best, 1 if renormalise else 0,
                                          float(scale), _stream(stream))
    if status:
        _check(status, "expert_route")
    return ids, weights


def expert_order(ids, E: int, out=None, stream=None):
    """(rows, offsets): the pairs (elements of the int32 ids [T, top_k]) by expert, int32 [T * top_k] with -1 behind the
    last, and where each expert's begin, int32 [E + 1]. Ids outside 0..E-1 have no expert. out: (rows, offsets) to write to."""
    torch = _torch or _load_torch()
    _here(ids)
    R = ids.numel()
    _ints("R E", R, E)
    pi = _weights("ids", ids, R, torch.int32)
    if out is None:
        rows, offsets = (_empty((R,), torch.int32, ids.device, stream), _empty((E + 1,), torch.int32, ids.device, stream))
    else:
        rows, offsets = out
        _here(rows, offsets)
        _packed("rows", rows, (R,), torch.int32)
        _packed("offsets", offsets, (E + 1,), torch.int32)
    status = (_lib or lib()).expert_order(pi, rows.data_ptr(), offsets.data_ptr(), R, E, _stream(stream))
    if status:
        _check(status, "expert_order")
    return rows, offsets


def w4a16_experts(A, W, scales, rows, offsets, N: int, K: int, global_scales=None, gated: bool = False, out=None,
                  stream=None):
    """C[p] = A[p / slots] @ dequant(W[e])^T for every pair p of each expert e, bfloat16 [R, N]; gated: silu(gate) * up of
    its two halves, [R, N / 2]. A is bfloat16 [R, K], or [T, K] with R = T * slots; W and scales hold E W4A16 matrices
    [N, K], global_scales their float32 scales [E]; rows and offsets are expert_order's. Rows of pairs without an expert
    are not written: a new out holds anything there."""
    torch = _torch or _load_torch()
    _here(A, W, scales, rows, offsets, global_scales, out)
    T, lda = _rows(A, K)
    E, R = offsets.numel() - 1, rows.numel()
    if E < 1:
        raise ValueError("offsets must hold E + 1 values")
    slots = R // T if T else 1
    if R != T * slots or slots < 1 and T:
        raise ValueError(f"{R} pairs are not a multiple of the {T} rows of A")
    _ints("T slots E N K", T, slots, E, N, K)
    pr, po = _packed("rows", rows, (R,), torch.int32), _packed("offsets", offsets, (E + 1,), torch.int32)
    pw, ps = _weights("W", W, E * N * (K // 2), torch.uint8), _weights("scales", scales, E * N * (K // 16), torch.uint8)
    pg = None if global_scales is None else _packed("global_scales", global_scales, (E,), torch.float32)
    if gated and N % 2:
        raise ValueError(f"N={N} must be even, gate and up")
    C, ldc = _gemm_out(A, R, N // 2 if gated else N, out, stream)
    L = _lib or lib()
    need = L.w4a16_experts_workspace(T, slots, E, N, K)
    work = _empty((need,), torch.uint8, A.device, stream) if need else None
    status = L.w4a16_experts(A.data_ptr(), lda, pw, ps, pg, pr, po, C.data_ptr(), ldc, T, slots, E, N, K, 1 if gated else 0,
                             _ptr(work), _stream(stream))
    if status:
        _check(status, "w4a16_experts")
    return C


def _rows_of(name, t, shape, y):
    """The pitch of rows of a given shape with the type of y."""
    if not t.is_cuda:
        raise ValueError("all tensors must be CUDA tensors (no CPU fallback)")
    stride = t.stride()
    if t.dtype is not y.dtype or t.shape != shape or (stride[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name} must be {list(shape)} of y's type, with unit column stride")
    ld = stride[0] if shape[0] > 1 else shape[1]
    if ld > _INT_MAX:
        _too_far(name, ld)
    return ld


def expert_combine(y, weights, ids, E: int, residual=None, out=None, stream=None):
    """[T, H]: residual + the sum over the slots of weights[t, s] * y[t * slots + s], in y's type (bfloat16, float16 or
    float32); y [T * slots, H], float32 weights and int32 ids [T, slots]. Rows whose id is outside 0..E-1 are not read.
    out may be the residual."""
    torch = _torch or _load_torch()
    _here(y, weights, ids, residual, out)
    ldy, dt, R, H = _typed_rows("y", y)
    of = weights.shape
    if len(of) != 2 or of[0] * of[1] != R:
        raise ValueError(f"weights must be [T, slots] with T * slots = {R}")
    T, slots = of
    _ints("T slots E H", T, slots, E, H)
    pw, pi = _packed("weights", weights, (T, slots), torch.float32), _packed("ids", ids, (T, slots), torch.int32)
    shape, pr, ldr = (T, H), None, 0
    if residual is not None:
        pr, ldr = residual.data_ptr(), _rows_of("residual", residual, shape, y)
    if out is None:
        out, ldo = _empty(shape, y.dtype, y.device, stream), H
    else:
        ldo = ldr if out is residual else _rows_of("out", out, shape, y)
    status = (_lib or lib()).expert_combine(y.data_ptr(), ldy, pw, pi, E, pr, ldr, out.data_ptr(), ldo, dt, T, slots, H,
                                            _stream(stream))
    if status:
        _check(status, "expert_combine")
    return out


def _deq_out(W, N, K, out, stream):
    if out is None:
        out = _empty((N, K), (_torch or _load_torch()).float32, W.device, stream)
    return out


def q2_dequant(W, N: int, K: int, out=None, stream=None):
    _need_cuda(W, out)
    o = _deq_out(W, N, K, out, stream)
    _check(lib().q2_dequant(_ptr(W), _ptr(o), N, K, _stream(stream)), "q2_dequant")
    return o


def w4a16_dequant(W, scales, N: int, K: int, global_scale: float = 1.0, out=None, stream=None):
    _need_cuda(W, scales, out)
    o = _deq_out(W, N, K, out, stream)
    _check(lib().w4a16_dequant(_ptr(W), _ptr(scales), float(global_scale), _ptr(o), N, K,
                               _stream(stream)), "w4a16_dequant")
    return o


def w8a16_dequant(W, scales, N: int, K: int, out=None, stream=None):
    _need_cuda(W, scales, out)
    o = _deq_out(W, N, K, out, stream)
    _check(lib().w8a16_dequant(_ptr(W), _ptr(scales), _ptr(o), N, K, _stream(stream)),
           "w8a16_dequant")
    return o


def row_chunks(M: int, K: int, N: int, max_rows: int):
    """Host-side row chunking: list of (a_byte_offset, c_byte_offset, rows)."""
    cap = max(1, (M + max(max_rows, 1) - 1) // max(max_rows, 1))
    buf = (ctypes.c_longlong * (3 * cap))()
    n = lib().wqp_row_chunks(M, K, N, max_rows, buf, cap)
    if n < 0:
        raise ValueError("invalid row_chunks arguments")
    return [(buf[3 * i], buf[3 * i + 1], buf[3 * i + 2]) for i in range(n)]


def set_pdl(enable: bool) -> bool:
    """Process-wide programmatic-dependent-launch policy; returns the old one. With it on, weights may be
    read before earlier launches have finished: make the first launch after writing weights without it."""
    return bool(lib().wqp_set_pdl(1 if enable else 0))


def get_device_error() -> int:
    """Read and clear the device error word (synchronises the device)."""
    return lib().wqp_get_device_error()


def selftest_wait_timeout(limit_us: int = 2000, stream=None) -> None:
    """Launch the failure-path self-test: a kernel whose bounded wait on a
    barrier nothing completes gives up after limit_us microseconds and records
    the timeout in the device error word (read it with get_device_error())."""
    _check(lib().wqp_selftest_wait_timeout(int(limit_us), _stream(stream)), "wqp_selftest_wait_timeout")
