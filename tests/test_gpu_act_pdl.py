"""The quantised-activation entries launched with programmatic dependent launch: every call of a chain reads what the
call before it wrote, into the same buffers with other inputs each time, so that a value left from the pass before
shows. Each pass is compared, bit for bit, with the same calls made without PDL."""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_packed_gb300 as wqp
from tests import _gpu as G

pytestmark = pytest.mark.gpu
DEV = "cuda"
PASSES = 6


@pytest.fixture(autouse=True)
def _pdl_off():
    old = wqp.set_pdl(False)
    yield
    wqp.set_pdl(old)
    assert wqp.get_device_error() == 0


def passes(M, K):
    g = torch.Generator(device=DEV).manual_seed(M + K)
    return [torch.randn((M, K), generator=g, device=DEV).mul_(2.0 ** (i % 3)).bfloat16() for i in range(PASSES)]


def w8_weights(N, K, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = (torch.randn((N, K), generator=g, device=DEV) * 20).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return w, torch.rand(((N + 127) // 128, K // 128), generator=g, device=DEV) + 0.5


def assert_same_under_pdl(chain, inputs):
    """chain(x) -> tensors, its own buffers."""
    want = [[t.clone() for t in chain(x)] for x in inputs]
    torch.cuda.synchronize()
    for _ in range(3):
        for x, w in zip(inputs, want):
            wqp.set_pdl(True)
            got = chain(x)
            wqp.set_pdl(False)
            got = [t.clone() for t in got]
            assert all(torch.equal(a, b) for a, b in zip(got, w))


@pytest.mark.parametrize("M", [1, 40, 3000])
def test_quantise_then_unpack(M):
    K = 5120
    codes, scales = wqp.w4_quantize(torch.zeros(M, K, device=DEV))
    values = torch.empty((M, K), device=DEV)

    def chain(x):
        wqp.w4_quantize(x, 0.03, out=(codes, scales))
        return codes, scales, wqp.w4a16_dequant(codes, scales, M, K, 0.03, out=values)

    assert_same_under_pdl(chain, passes(M, K))


@pytest.mark.parametrize("M", [1, 40, 700])
def test_norm_then_unpack_then_product(M):
    """The unpacking in between has nothing to do with the rows: the product has to wait for the norm all the same."""
    N, K = 640, 5120
    w = torch.ones(K, dtype=torch.bfloat16, device=DEV)
    w8, s8 = w8_weights(N, K, 1)
    small, ss = w8_weights(128, 128, 2)
    q2 = torch.zeros(8 * 34 * 8, dtype=torch.uint8, device=DEV)
    codes, scales, h = wqp.rms_norm_a8(passes(M, K)[0], w, 1e-6, residual=passes(M, K)[1])
    u = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
    v, v2 = torch.empty((128, 128), device=DEV), torch.empty((8, 1024), device=DEV)

    def chain(x):
        wqp.rms_norm_a8(x, w, 1e-6, residual=x, residual_out=h, out=(codes, scales))
        wqp.w8a16_dequant(small, ss, 128, 128, out=v)
        wqp.q2_dequant(q2, 8, 1024, out=v2)
        return wqp.w8a8_gemm(codes, scales, w8, s8, N, K, out=u), h, v

    assert_same_under_pdl(chain, passes(M, K))


@pytest.mark.parametrize("M", [1, 24, 64, 100, 300])
@pytest.mark.parametrize("fmt", [4, 8])
def test_quantise_then_product(fmt, M):
    """The rows' codes and scales are written by the kernel just before, over those of the pass before; M over the
    kernels' ranges, with K split (640 columns) and not."""
    K = 5120
    first = passes(M, K)[0]
    for N in (640, 20480):
        u = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
        if fmt == 4:
            w, sw = wqp.w4_quantize(torch.randn((N, K), generator=torch.Generator(device=DEV).manual_seed(N), device=DEV), 0.002)
            codes, scales = wqp.w4_quantize(first, 0.01)

            def chain(x):
                wqp.w4_quantize(x, 0.01, out=(codes, scales))
                return codes, scales, wqp.w4a4_gemm(codes, scales, w, sw, N, K, 0.01, 0.002, out=u)
        else:
            w, sw = w8_weights(N, K, N)
            codes, scales = wqp.a8_quantize(first)

            def chain(x):
                wqp.a8_quantize(x, out=(codes, scales))
                return codes, scales, wqp.w8a8_gemm(codes, scales, w, sw, N, K, out=u)

        assert_same_under_pdl(chain, passes(M, K))


WEIGHT_ONLY = {
    "q2": (wqp.q2_gemv, wqp.q2_gemm_tc, wqp.q2_gemm_mma),
    "w4": (wqp.w4a16_gemv, wqp.w4a16_gemm_tc, wqp.w4a16_gemm_mma),
    "w8": (wqp.w8a16_gemm, wqp.w8a16_gemm_tc, wqp.w8a16_gemm_mma),
}


@pytest.mark.parametrize("M", [1, 5, 16])
@pytest.mark.parametrize("N,K", [(640, 5120), (1000, 1024)])
@pytest.mark.parametrize("fmt", sorted(WEIGHT_ONLY))
def test_norm_then_weight_only_products(fmt, N, K, M):
    """The norm's BF16 rows are the next kernel's activations, which it has to read as they were just written."""
    d = G.make(fmt, 1, N, K, seed=77)
    weights = (d["dW"],) if fmt == "q2" else (d["dW"], d["dS"])
    w = torch.ones(K, dtype=torch.bfloat16, device=DEV)
    y = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
    outs = [torch.empty((M, N), dtype=torch.bfloat16, device=DEV) for _ in WEIGHT_ONLY[fmt]]

    def chain(x):
        for call, out in zip(WEIGHT_ONLY[fmt], outs):
            wqp.rms_norm(x, w, 1e-6, out=y)
            call(y, *weights, N, K, out=out)
            x = x * 1.5 - 0.25
        return outs

    assert_same_under_pdl(chain, passes(M, K))
