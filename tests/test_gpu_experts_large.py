"""The experts' entries on buffers beyond 2^31 elements (weights, rows, workspace, outputs, logits), and each step of a block
from the logits on. Bounds and plain forms are tests/test_gpu_experts.py's."""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_packed_gb300 as wqp
from tests.test_gpu_experts import DEV, U, Block, experts64, gen, make_experts, order_plain, route64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert wqp.get_device_error() == 0


def far_rows(rows, cols, pitch, dtype, fill=None):
    """[rows, cols] whose rows are `pitch` elements apart."""
    buf = torch.empty((rows - 1) * pitch + cols + 8, dtype=dtype, device=DEV)
    if fill is not None:
        buf.as_strided((rows, cols + 8), (pitch, 1)).fill_(fill)
    return buf.as_strided((rows, cols), (pitch, 1))


@pytest.mark.parametrize("gated", [False, True])
def test_a_decode_batch_and_the_last_of_many_experts(gated):
    """About a pair an expert and K = 5120, which goes by the weights' size to the kernel for many rows: its maps of codes and
    scales beyond 2^31 bytes and 2^31 elements."""
    E, N, K, T = 220, 4096, 5120, 64
    g = gen(20)
    w = torch.zeros((E, N, K // 2), dtype=torch.uint8, device=DEV)
    s = torch.zeros((E, N, K // 16), dtype=torch.uint8, device=DEV)
    w[-1] = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    s[-1] = 0x28
    a = torch.randn((T, K), generator=g, device=DEV).bfloat16()
    ids = torch.arange(T, dtype=torch.int32, device=DEV).view(T, 1) * 3
    ids[5] = ids[40] = ids[63] = E - 1
    got = wqp.w4a16_experts(a, w, s, *wqp.expert_order(ids, E), N, K, gated=gated).double().cpu()
    hit = [5, 40, 63]
    want, tol, _ = experts64(a[hit], w[-1:], s[-1:], None, torch.zeros(3, 1, dtype=torch.int32), gated, 1)
    assert ((got[hit] - want).abs() <= tol).all()
    rest = torch.ones(T, dtype=torch.bool)
    rest[hit] = False
    assert (got[rest] == 0).all()


@pytest.mark.parametrize("T,pitch", [(5, 2 ** 29 + 64), (72, 2 ** 25 + 64)])    # few pairs an expert, many
@pytest.mark.parametrize("gated", [False, True])
def test_rows_and_outputs_far_apart(T, pitch, gated):
    """Rows of A and of C whose distance from their base passes 2^31 elements."""
    E, N, K = 3, 40, 256
    g = gen(21)
    w, s, gs = make_experts(E, N, K, 22)
    a = far_rows(T, K, pitch, torch.bfloat16)
    a.copy_(torch.randn((T, K), generator=g, device=DEV))
    assert (T - 1) * pitch > 2 ** 31
    ids = torch.randint(0, E, (T, 1), generator=g, device=DEV, dtype=torch.int32)
    F = N // 2 if gated else N
    out = far_rows(T, F, pitch, torch.bfloat16, fill=-5.0)
    got = wqp.w4a16_experts(a, w, s, *wqp.expert_order(ids, E), N, K, gs, gated, out=out).double().cpu()
    want, tol, _ = experts64(a.contiguous(), w, s, gs, ids, gated, 1)
    assert ((got - want).abs() <= tol).all()
    assert (out.as_strided((T, 8), (pitch, 1), out.storage_offset() + F) == -5).all()


def test_a_workspace_beyond_2_31_elements():
    """2^18 pairs of K = 8320: the rows in the pairs' order pass 2^31 elements, the last pairs' among them."""
    T, k, E, N, K = 2 ** 15, 8, 4, 16, 8320
    g = gen(23)
    w, s, gs = make_experts(E, N, K, 24)
    a = torch.randn((T, K), generator=g, device=DEV).bfloat16()
    ids = torch.randint(0, E, (T, k), generator=g, device=DEV, dtype=torch.int32)
    rows, offsets = wqp.expert_order(ids, E)
    got = wqp.w4a16_experts(a, w, s, rows, offsets, N, K, gs)
    some = rows[[0, 1, 2 ** 17, 2 ** 18 - 9000, 2 ** 18 - 2, 2 ** 18 - 1]].long()
    want, tol, _ = experts64(a[some // k], w, s, gs, ids.view(-1)[some].view(-1, 1), False, 1)
    assert ((got[some].double().cpu() - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_combine_far_apart(dtype):
    T, k, H, pitch, E = 3, 2, 48, 2 ** 29 + 32, 4
    g = gen(25)
    y, res, out = far_rows(T * k, H, pitch, dtype), far_rows(T, H, pitch * 2, dtype), far_rows(T, H, pitch * 2, dtype, fill=-5.0)
    y.copy_(torch.randn((T * k, H), generator=g, device=DEV))
    res.copy_(torch.randn((T, H), generator=g, device=DEV))
    ids = torch.randint(0, E, (T, k), generator=g, device=DEV, dtype=torch.int32)
    weights = torch.rand((T, k), generator=g, device=DEV)
    assert (T - 1) * pitch * 2 > 2 ** 31
    got = wqp.expert_combine(y, weights, ids, E, residual=res, out=out)
    assert torch.equal(got, wqp.expert_combine(y.contiguous(), weights, ids, E, residual=res.contiguous()))
    assert (out.as_strided((T, 8), (pitch * 2, 1), out.storage_offset() + H) == -5).all()


def test_route_far_apart():
    T, E, pitch = 5, 96, 2 ** 29 + 1
    x = far_rows(T, E, pitch, torch.bfloat16)
    x.copy_(torch.randn((T, E), generator=gen(26), device=DEV))
    assert (T - 1) * pitch > 2 ** 31
    got, want = wqp.expert_route(x, 7), wqp.expert_route(x.contiguous(), 7)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T", [1, 19, 260])
def test_block_from_its_logits(T):
    """What test_gpu_experts.py's test_block takes as given: the block's experts, weights and order."""
    b = Block(512, 256, 16, 4)
    x = torch.randn((T, b.H), generator=gen(T), device=DEV).bfloat16()
    logits = x.float() @ b.router
    ids, weights = wqp.expert_route(logits, b.k, "sigmoid", b.bias, 4, 2)
    assert all(torch.equal(p, q) for p, q in zip(b(x, x)[:2], (ids, weights)))
    want, w = route64(logits, b.k, "sigmoid", b.bias, 4, 2, 2, True, 1.0)
    span = 2 * float(logits.abs().max())
    assert torch.equal(ids.cpu(), want) and ((weights.double().cpu() - w).abs() <= (64 + 2 * span) * U * w).all()
    rows, offsets = wqp.expert_order(ids, b.E)
    want_rows, want_offsets = order_plain(ids, b.E)
    assert rows.tolist() == want_rows and offsets.tolist() == want_offsets
