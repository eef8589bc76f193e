"""Calls on a stream other than the current one, whose outputs and dropped intermediates share the allocator with work
on the current stream."""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_packed_gb300 as wqp

pytestmark = pytest.mark.gpu
DEV = "cuda"


def pool_of(t):
    """The stream in whose pool a tensor's block lies."""
    at = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's")


@pytest.mark.parametrize("as_handle", [False, True])
def test_a_chain_on_a_side_stream_beside_work_on_the_current_one(as_handle):
    """Norm, 8-bit product, 4-bit rows, 4-bit product: what the chain drops on the way is of the sizes that the current
    stream allocates and fills meanwhile."""
    M, K, N = 512, 5120, 2048
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn((M, K), generator=g, device=DEV).bfloat16()
    norm = torch.ones(K, dtype=torch.bfloat16, device=DEV)
    w8, s8 = wqp.a8_quantize(torch.randn((N, K), generator=g, device=DEV) / 64)
    s8 = s8[::128].contiguous()
    w4, s4 = wqp.w4_quantize(torch.randn((K, N), generator=g, device=DEV) / 64, 0.001)

    def chain(stream=None):
        c, s, h = wqp.rms_norm_a8(x, norm, 1e-6, residual=x, stream=stream)
        u = wqp.w8a8_gemm(c, s, w8, s8, N, K, stream=stream)
        q, qs = wqp.w4_quantize(u, 0.01, stream=stream)
        return wqp.w4a4_gemm(q, qs, w4, s4, K, N, 0.01, 0.001, stream=stream), h

    want = chain()
    assert want[0].isfinite().all()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    stream = side.cuda_stream if as_handle else side
    for _ in range(20):
        got = chain(stream)
        fill = [torch.full(t.shape, float("nan"), dtype=t.dtype, device=DEV) for t in (*got, x)]
        fill += [torch.full((M, k), 0xFF, dtype=torch.uint8, device=DEV) for k in (K, N // 2, N // 16)]
        assert {pool_of(t) for t in got} == {side.cuda_stream}
        assert {pool_of(t) for t in fill} == {torch.cuda.current_stream().cuda_stream}
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del got, fill
        side.wait_stream(torch.cuda.current_stream())


def test_the_default_stream_passed_as_a_handle():
    x = torch.ones(4, 256, dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        codes, scales = wqp.a8_quantize(x, stream=0)
    torch.cuda.synchronize()
    assert {pool_of(codes), pool_of(scales)} == {torch.cuda.default_stream().cuda_stream}
    assert (codes == 0x7E).all()
