"""The experts' entries where values leave FP32's range on the way, against 64-bit forms.

Routing, u = 2^-24. sigmoid(l) = e^min(l, 0) / (1 + e^-|l|), and its quotient by the largest taken one's has the difference of
the two exponents: an argument that is off by u |x|, exponentials of 2 ulp (4 u), a sum of at most 32 with 5 roundings on
any path, three divisions or products: relatively (64 + 2 |x|) u, |x| at most twice the largest logit. Below FP32's normal
range the exponential is off by 2 * 2^-149 and each step rounds to 2^-150; the sum is 1/2 at least, so all in all by less than
2^-146 before the scale.
"""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_packed_gb300 as wqp
from tests.test_gpu_experts import DEV, INF, U, gen

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
