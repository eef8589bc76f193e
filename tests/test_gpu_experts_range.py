"""The experts' entries where values leave FP32's range on the way, against 64-bit forms.

Routing, u = 2^-24. sigmoid(l) = e^min(l, 0) / (1 + e^-|l|), and its quotient by the largest taken one's has the difference of
the two exponents: an argument that is off by u |x|, exponentials of 2 ulp (4 u), a sum of at most 32 with 5 roundings on
any path, three divisions or products: relatively (64 + 2 |x|) u, |x| at most twice the largest logit. Below FP32's normal
range the exponential is off by 2 * 2^-149 and each step rounds to 2^-150; the sum is 1/2 at least, so all in all by less than
2^-146 before the scale.

silu(g) = g sigmoid(g) through t = e^-|g|, in both product kernels: t is off by 2 ulp (4 u; 2 u of the result again through
1 + t), g t and 1 + t by u each, the quotient by 2 ulp (4 u) and its product with the other half by u: 13 u, and where t is
below FP32's normal range 2^-148 of it, and 2^-150 of g t. Then half a step of BF16.
"""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_packed_gb300 as wqp
from tests.test_gpu_experts import DEV, INF, U, gen, unpack

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert wqp.get_device_error() == 0


# ---------------------------------------------------------------- routing
def check_sigmoid_weights(x, ids, w, renormalise, scale):
    """The weights of the experts taken, from logarithms, so that no quotient of vanishing scores is lost."""
    x, ids = x.double().cpu(), ids.long().cpu()
    l = torch.where(ids >= 0, torch.nn.functional.logsigmoid(x.gather(1, ids.clamp_min(0))), -INF)
    if renormalise:
        l = l - torch.where((ids >= 0).any(1, keepdim=True), torch.logsumexp(l, 1, keepdim=True), 0.0)
    want = l.exp() * scale
    span = 2 * float(torch.where(x.isinf(), 0.0, x).abs().amax())
    off = (w.double().cpu() - want).abs()
    assert (off <= (64 + 2 * span) * U * want.abs() + 2.0 ** -146 * abs(scale)).all(), (float(off.max()), w, want)


@pytest.mark.parametrize("logits", [[-79, -89], [-79.5, -88, -89, -90, -100, -103], [-50, -88.5, -95, -120], [-20, -87, -88.7, -88.8, -110],
                                    [-3, -89, -102], [0, -104], [30, -95, -101], [-81, -90], [-88, -88, -89], [INF, -90, -100], [-5000, -5001]])
@pytest.mark.parametrize("renormalise", [False, True])
def test_sigmoid_weights_far_below_zero(logits, renormalise):
    x = torch.tensor([logits], dtype=torch.float32, device=DEV)
    ids, w = wqp.expert_route(x, len(logits), "sigmoid", renormalise=renormalise, scale=1.5)
    assert ids.tolist() == [list(range(len(logits)))]
    check_sigmoid_weights(x, ids, w, renormalise, 1.5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("shift,spread", [(-90, 1), (-90, 10), (-60, 20), (-40, 60), (0, 100)])
@pytest.mark.parametrize("renormalise", [False, True])
def test_sigmoid_weights_of_experts_that_the_bias_chooses(dtype, shift, spread, renormalise):
    """With a bias that outweighs the scores, the taken experts' logits lie anywhere."""
    g = gen(spread - shift)
    x = (torch.randn((50, 64), generator=g, device=DEV) * spread + shift).to(dtype)
    x[torch.rand((50, 64), generator=g, device=DEV) < 0.3] = -INF
    x[3] = -INF
    bias = torch.randn(64, generator=g, device=DEV) * 100
    ids, w = wqp.expert_route(x, 12, "sigmoid", bias=bias, renormalise=renormalise, scale=-2.5)
    live = torch.where(x.isneginf(), -INF, torch.sigmoid(x.double()) + bias.double())
    best = torch.sort(live, dim=1, descending=True, stable=True)
    assert torch.equal(ids, torch.where(best.values > -INF, best.indices, -1)[:, :12].int())
    check_sigmoid_weights(x, ids, w, renormalise, -2.5)


# ---------------------------------------------------------------- silu
def bf16_step(v):
    """BF16's step at the magnitude v (64 bits)."""
    return torch.exp2(torch.floor(torch.log2(v.clamp_min(2.0 ** -126))) - 7)


@pytest.mark.parametrize("T", [4, 200])                      # few pairs an expert, many
@pytest.mark.parametrize("reach", [1, 20, 60, 86, 104])
def test_silu(T, reach):
    """Gates and ups that are exact in FP32: one product each, of activations within a factor of 2^31, which FP16 takes as they
    are. What is left is silu's own error and one rounding. The gates reach down to where e^g leaves FP32's normal numbers,
    the ups bring the outputs back."""
    E, N, K = 1, 4096, 128
    g = gen(T + reach)
    F = N // 2
    w, s = torch.zeros((E, N, K // 2), dtype=torch.uint8, device=DEV), torch.zeros((E, N, K // 16), dtype=torch.uint8, device=DEV)
    w[0, :F, 0] = torch.randint(1, 8, (F,), generator=g, device=DEV, dtype=torch.uint8)      # gate: element 0
    w[0, F:, 8] = torch.randint(1, 8, (F,), generator=g, device=DEV, dtype=torch.uint8)      # up: element 16
    s[0, :F, 0] = torch.randint(0x30, 0x48, (F,), generator=g, device=DEV, dtype=torch.uint8)
    s[0, F:, 1] = torch.randint(0x30, 0x48, (F,), generator=g, device=DEV, dtype=torch.uint8)
    value = unpack(w, s)[0]
    a = torch.zeros((T, K), dtype=torch.bfloat16, device=DEV)
    a[:, 0] = (torch.rand(T, generator=g, device=DEV) * 0.98 + 0.02) * reach / float(value[:F, 0].max())
    a[:, 0] *= torch.where(torch.rand(T, generator=g, device=DEV) < 0.8, -1.0, 1.0)
    a[0, 0] = -reach / float(value[:F, 0].max())             # to the end of the reach
    a[:, 16] = (torch.rand(T, generator=g, device=DEV) + 0.5) * 2.0 ** (20 if reach > 60 else 0)
    ids = torch.zeros((T, 1), dtype=torch.int32, device=DEV)
    got = wqp.w4a16_experts(a, w, s, *wqp.expert_order(ids, E), N, K, gated=True).double().cpu()
    x = a.double().cpu()
    assert float((x[:, 16] / x[:, 0].abs()).max()) < 2.0 ** 31
    gate, up = x[:, :1] * value[:F, 0], x[:, 16:17] * value[F:, 16]
    want = gate * torch.sigmoid(gate) * up
    off = 13 * U * want.abs() * (1 + 2.0 ** -16) + (gate.abs() * 2.0 ** -148 + 2.0 ** -150) * up.abs()
    tol = off + bf16_step(want.abs() + off) / 2
    bad = (got - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), gate[bad][:4], up[bad][:4], got[bad][:4], want[bad][:4])
