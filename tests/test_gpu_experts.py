"""The experts' entries on the GPU against plain 64-bit forms.

Tolerances, each from the arithmetic alone (u = 2^-24):

* Routing. The order is exact. A score is an exponential (2 ulp, 4 u of it) of an argument that is off by u |x|, over a
  sum of at most 37 roundings on any path, and three further operations: relatively (64 + 2 |x|) u, |x| the span of the
  logits; values below FP32's normal range are off by 2^-149 as well.
* Products. All products are exact. A sum of K of them goes through K / 16 MMA steps, K / 128 additions and 8 more, each
  rounded or cut to 2^-23 of the largest partial sum, which is at most S, the sum of magnitudes; an activation below 2^-31
  of its block's largest is off by 2^-39 of that: (K / 16 + K / 128 + 16) 2^-23 S and less than 2^-24 S besides, in all
  (K / 8 + 32) 2^-23 S. BF16 adds 2^-8. silu(g) * v: |silu'| <= 1.1, and 8 u of the result for its own operations.
  Where all partial sums are integers below 2^24 the result is the exact one.
* Combining. At most 34 additions of products: 35 u of the sum of magnitudes, and the rounding to the output's type.
"""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_packed_gb300 as wqp

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
INF, NAN = float("inf"), float("nan")
TYPES = [torch.bfloat16, torch.float16, torch.float32]
E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert wqp.get_device_error() == 0


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


# ---------------------------------------------------------------- routing
def route64(logits, k, scoring, bias, groups, top_groups, group_best, renormalise, scale):
    """Token by token, in Python's own floats' precision: (ids, weights)."""
    T, E = logits.shape
    x = logits.double().cpu()
    s = torch.sigmoid(x) if scoring == "sigmoid" else torch.softmax(torch.where(x.isneginf().all(1, keepdim=True), 0.0, x), 1)
    s = torch.where(x.isneginf(), 0.0, s)
    c = x if bias is None else torch.where(x.isneginf(), -INF, s + bias.double().cpu())
    ids = torch.full((T, k), -1, dtype=torch.int32)
    w = torch.zeros(T, k, dtype=torch.float64)
    for t in range(T):
        key = c[t].tolist()
        if groups > 1:
            size, base = E // groups, (s[t] if bias is None and group_best == 2 else c[t]).tolist()
            scores = []
            for g in range(groups):
                live = sorted((base[i] for i in range(g * size, (g + 1) * size) if key[i] > -INF), reverse=True)
                scores.append(sum(live[:group_best]) if live else -INF)
            stay = sorted(range(groups), key=lambda g: (-scores[g], g))[:top_groups]
            key = [v if i // size in stay else -INF for i, v in enumerate(key)]
        order = sorted((i for i in range(E) if key[i] > -INF), key=lambda i: (-key[i], i))[:k]
        ids[t, :len(order)] = torch.tensor(order, dtype=torch.int32)
        got = s[t, order]
        if renormalise and len(order):
            # Relative to the largest taken, so that 64 bits hold a quotient of vanishing exponentials too.
            if scoring == "softmax":
                got = torch.softmax(x[t, order], 0)
            else:
                got = got / got.sum()
        w[t, :len(order)] = got
    return ids, w * scale


def check_route(logits, k, scoring="softmax", bias=None, groups=1, top_groups=1, group_best=2, renormalise=True, scale=1.0):
    T, E = logits.shape
    ids, weights = wqp.expert_route(logits, k, scoring, bias, groups, top_groups, group_best, renormalise, scale)
    want, w = route64(logits, k, scoring, bias, groups, top_groups, group_best, renormalise, scale)
    assert ids.dtype == torch.int32 and ids.shape == weights.shape == (T, k)
    assert torch.equal(ids.cpu(), want)
    x = logits.double().cpu()
    span = float(torch.where(x.isinf(), 0.0, x).abs().amax()) * 2 if T else 0.0
    off = (weights.double().cpu() - w).abs()
    assert (off <= (64 + 2 * span) * U * w.abs() + 2.0 ** -140 * abs(scale)).all(), float((off / w.abs().clamp_min(1e-300)).amax())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 2, 2), (5, 31, 4), (4, 33, 32), (9, 64, 8), (7, 65, 6), (33, 128, 8), (6, 257, 1), (5, 512, 10),
                                   (3, 1000, 32), (2, 1024, 8)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_plain(dtype, T, E, k, scoring):
    g = gen(T * E + k)
    x = (torch.randn((T, E + 3), generator=g, device=DEV) * 3).to(dtype)[:, :E]
    check_route(x, k, scoring)
    check_route(x, k, scoring, renormalise=False, scale=2.5)
    check_route(x, k, scoring, bias=torch.randn(E, generator=g, device=DEV) * 0.1)


@pytest.mark.parametrize("E,groups,top_groups,k", [(8, 8, 3, 3), (32, 32, 5, 5), (24, 3, 2, 16), (256, 8, 4, 8), (60, 5, 1, 12), (1024, 32, 31, 32), (40, 20, 20, 7),
                                                  (64, 2, 2, 6)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_best", [1, 2])
@pytest.mark.parametrize("biased", [False, True])
def test_route_groups(E, groups, top_groups, k, scoring, group_best, biased):
    g = gen(E + groups)
    x = torch.randn((21, E), generator=g, device=DEV) * 2
    bias = torch.randn(E, generator=g, device=DEV) * 0.2 if biased else None
    check_route(x, k, scoring, bias, groups, top_groups, group_best)
    x[torch.rand((21, E), generator=g, device=DEV) < 0.7] = -INF      # groups with one expert and with none
    x[4] = -INF
    check_route(x, k, scoring, bias, groups, top_groups, group_best)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (4, 2)])
@pytest.mark.parametrize("biased", [False, True])
def test_route_ties_go_to_the_lower_index(scoring, groups, top_groups, biased):
    g = gen(5)
    x = torch.randint(-1, 2, (40, 64), generator=g, device=DEV).bfloat16()
    bias = torch.randint(0, 2, (64,), generator=g, device=DEV).float() * 0.25 if biased else None
    check_route(x, 12, scoring, bias, groups, top_groups)
    check_route(torch.zeros(3, 64, device=DEV), 12, scoring, torch.zeros(64, device=DEV), groups, top_groups)
    check_route(torch.tensor([[-0.0, 0.0] * 32], device=DEV), 12, scoring, None, groups, top_groups)


@pytest.mark.parametrize("E,groups,top_groups", [(64, 1, 1), (64, 4, 2), (512, 8, 3)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_choices_that_fp32_cannot_tell_apart(E, groups, top_groups, scoring):
    """The biases make up for the scores up to FP32's last bit, so every choice lies within some 2^-24 of every other."""
    x = torch.randn((1, E), generator=gen(E), device=DEV)
    s = torch.sigmoid(x.double()) if scoring == "sigmoid" else torch.softmax(x.double(), 1)
    bias = (1.0 - s[0]).float()
    for shift in (0.0, 2.0 ** -20, 1.0):
        check_route(x + shift, 8, scoring, bias, groups, top_groups, 2)
        check_route(x + shift, 8, scoring, bias, groups, top_groups, 1)


@pytest.mark.parametrize("E,groups,top_groups", [(64, 4, 2), (256, 8, 4), (96, 32, 7), (120, 5, 3)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_best", [1, 2])
def test_route_groups_that_fp32_cannot_tell_apart(E, groups, top_groups, scoring, group_best):
    """Every group has two experts that stand out and lie within FP32's last bits of the other groups'; biases of +-infinity."""
    g = gen(E + groups)
    x = torch.randn((40, E), generator=g, device=DEV)
    s = (torch.sigmoid(x.double()) if scoring == "sigmoid" else torch.softmax(x.double(), 1)).cpu()
    bias = torch.full((E,), -3.0)
    first = torch.arange(groups) * (E // groups)
    for at in (first, first + 1):
        bias[at] = (1.0 - s[0, at]).float()
    for shift in (0.0, 2.0 ** -22):
        check_route(x + shift, 3, scoring, bias.to(DEV), groups, top_groups, group_best)
    if group_best == 2:
        check_route(x[:1].expand(3, E).contiguous(), 2, scoring, None, groups, top_groups)
    bias[2::E // groups] = bias[2].item()                    # a third, far below
    bias[0] = bias[1] = bias[E - 1] = INF
    bias[3] = -INF
    check_route(x, 3, scoring, bias.to(DEV), groups, top_groups, group_best)


def test_route_far_logits():
    """Scores that vanish in FP32, and their quotients."""
    x = torch.zeros(4, 16, device=DEV)
    x[0] = -200.0 - torch.arange(16, device=DEV)
    x[1] = torch.linspace(-3e38, 3e38, 16, device=DEV)
    x[2, 0] = 500.0
    x[3] = 90.0 + torch.arange(16, device=DEV) * 0.5
    bias = torch.zeros(16, device=DEV)
    bias[12:] = 3.0                              # taken although their scores vanish
    ids, w = wqp.expert_route(x[2:3], 2, "softmax", bias=bias)
    assert ids.tolist() == [[12, 13]] and torch.allclose(w.cpu(), torch.tensor([[0.5, 0.5]]), rtol=1e-6)
    ids, w = wqp.expert_route(x, 4, "softmax")
    want = torch.softmax(x.double(), 1).topk(4, dim=1).values
    # Row 1 holds NaNs (the step of such a linspace passes FP32's range).
    assert torch.allclose(w.double(), want / want.sum(1, keepdim=True), rtol=1e-5, atol=1e-30, equal_nan=True)
    wide = torch.arange(-8, 8, device=DEV)[None] * 4e37
    for b in (None, bias):
        ids, w = wqp.expert_route(wide, 4, "softmax", bias=b)
        assert ids[0, 0] == 15 and w.tolist() == [[1.0, 0.0, 0.0, 0.0]]
    ids, w = wqp.expert_route(x[:1], 4, "sigmoid")
    assert ids.tolist() == [[0, 1, 2, 3]]
    assert torch.allclose(w.double().cpu(), torch.softmax(-torch.arange(4).double(), 0)[None], rtol=1e-6)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_route_nan_and_infinities(scoring, renormalise):
    x = torch.randn((6, 40), generator=gen(3), device=DEV)
    x[0, 7] = NAN
    x[1] = NAN
    x[2, 5] = INF
    x[3] = -INF
    x[4, 3:] = -INF
    bias = torch.zeros(40, device=DEV)
    for b in (None, bias):
        ids, w = wqp.expert_route(x, 5, scoring, bias=b, renormalise=renormalise)
        ids, w = ids.cpu(), w.cpu()
        assert w[0].isnan().all() and 7 not in ids[0].tolist() and (ids[0] >= 0).all()
        assert w[1].isnan().all() and (ids[1] == -1).all()
        if scoring == "softmax":
            assert w[2].isnan().all() and ids[2, 0] == 5
        else:
            assert ids[2, 0] == 5 and w[2].isfinite().all()
        assert (ids[3] == -1).all() and (w[3] == 0).all()
        assert sorted(ids[4, :3].tolist()) == [0, 1, 2] and (ids[4, 3:] == -1).all() and (w[4, 3:] == 0).all()
        assert w[4:].isfinite().all()
    bias[2] = NAN
    bias[3] = -INF
    bias[9] = INF
    ids, _ = wqp.expert_route(x[5:6], 32, scoring, bias=bias)
    assert ids[0, 0] == 9 and not {2, 3} & set(ids[0].tolist())


# ---------------------------------------------------------------- ordering
def order_plain(ids, E):
    flat = ids.cpu().view(-1).tolist()
    lists = [[i for i, e in enumerate(flat) if e == x] for x in range(E)] if E <= 64 else None
    if lists is None:
        lists = [[] for _ in range(E)]
        for i, e in enumerate(flat):
            if 0 <= e < E:
                lists[e].append(i)
    rows, offsets = [], [0]
    for at in lists:
        rows += at
        offsets.append(len(rows))
    return rows + [-1] * (len(flat) - len(rows)), offsets


@pytest.mark.parametrize("T,k", [(0, 4), (1, 1), (1, 8), (31, 1), (33, 3), (256, 8), (257, 8), (1000, 5), (2048, 1), (2049, 1), (8191, 8), (20011, 7)])
@pytest.mark.parametrize("E", [1, 7, 64, 256, 1024])
def test_order(T, k, E):
    ids = torch.randint(-2, E + 2, (T, k), generator=gen(T + E), device=DEV, dtype=torch.int32)
    rows, offsets = wqp.expert_order(ids, E)
    want_rows, want_offsets = order_plain(ids, E)
    assert offsets.tolist() == want_offsets and rows.tolist() == want_rows


@pytest.mark.parametrize("R", [40, 5000, 300001])
def test_order_of_one_expert_and_of_none(R):
    for e in (0, 5, 6, -1, 2 ** 31 - 1, -2 ** 31):
        ids = torch.full((R,), e, device=DEV, dtype=torch.int32)
        rows, offsets = wqp.expert_order(ids, 6)
        live = 0 <= e < 6
        assert offsets.tolist() == [0] * (e + 1 if live else 7) + [R] * (6 - e if live else 0)
        assert torch.equal(rows.cpu(), torch.arange(R, dtype=torch.int32) if live else torch.full((R,), -1, dtype=torch.int32))


# ---------------------------------------------------------------- products
def unpack(w, s):
    """[E, N, K] values of packed W4A16 matrices, in 64 bits."""
    c = w.cpu()
    v = E2M1[torch.stack((c & 15, c >> 4), 3).long()].view(*c.shape[:2], -1)
    return v * s.cpu().view(torch.float8_e4m3fn).double().repeat_interleave(16, 2)


def make_experts(E, N, K, seed):
    g = gen(seed)
    w = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = (torch.randn((E, N, K // 16), generator=g, device=DEV).abs() * 0.05).to(torch.float8_e4m3fn).view(torch.uint8)
    return w, s, 0.5 + torch.rand(E, generator=g, device=DEV)


def experts64(a, w, s, g, ids, gated, slots):
    """(values [R, N or N / 2], tolerance, live pairs)."""
    flat = ids.cpu().view(-1).long()
    E, K = w.shape[0], a.shape[1]
    v = unpack(w, s)
    g = torch.ones(E, dtype=torch.float64) if g is None else g.double().cpu()
    a = a.double().cpu()
    N = v.shape[1]
    u, S = torch.zeros(len(flat), N, dtype=torch.float64), torch.zeros(len(flat), N, dtype=torch.float64)
    live = (flat >= 0) & (flat < E)
    for e in flat[live].unique().tolist():
        at = (flat == e).nonzero().view(-1)
        x = a[at // slots]
        u[at] = x @ v[e].t() * g[e]
        S[at] = x.abs() @ v[e].abs().t() * g[e].abs()
    tol = (K / 8 + 32) * 2.0 ** -23 * S + 2 * U * u.abs()
    if gated:
        F = N // 2
        gate, up = u[:, :F], u[:, F:]
        act = gate * torch.sigmoid(gate)
        out = act * up
        tol = 1.1 * tol[:, :F] * (up.abs() + tol[:, F:]) + act.abs() * tol[:, F:] + 8 * U * out.abs()
        u = out
    return u, tol + 2.0 ** -8 * (u.abs() + tol) + 2.0 ** -134, live


def check_experts(T, k, E, N, K, gated, pairs=False, pad=0, seed=0, ids=None, a=None, globals_=True):
    g = gen(seed + T + N + K)
    w, s, gs = make_experts(E, N, K, seed)
    gs = gs if globals_ else None
    if ids is None:
        ids = torch.randint(-1, E, (T, k), generator=g, device=DEV, dtype=torch.int32)
    rows, offsets = wqp.expert_order(ids, E)
    M = T * k if pairs else T
    if a is None:
        a = torch.full((M, K + pad), 77.0, dtype=torch.bfloat16, device=DEV)
        a[:, :K] = torch.randn((M, K), generator=g, device=DEV) * torch.where(torch.rand(K, generator=g, device=DEV) < 0.02, 12.0, 1.0)
        a = a[:, :K]
    F = N // 2 if gated else N
    canvas = torch.full((T * k, F + pad + 3), -5.0, dtype=torch.bfloat16, device=DEV)
    out = canvas[:, 1:F + 1] if pad else canvas[:, :F]
    got = wqp.w4a16_experts(a, w, s, rows, offsets, N, K, gs, gated, out=out)
    assert got.data_ptr() == out.data_ptr()
    want, tol, live = experts64(a, w, s, gs, ids, gated, 1 if pairs else k)
    got = got.double().cpu()
    assert ((got - want).abs() <= tol)[live].all(), float(((got - want).abs() / tol)[live].max())
    assert (got[~live] == -5).all()
    canvas[:, 1 if pad else 0:][:, :F] = -5.0
    assert (canvas == -5).all()
    return a, w, s, gs, rows, offsets, ids


SHAPES = [
    # T, k, E, N, K: one pair; few; rows over several tiles of pairs; every tail of N; K over the warps and not
    (1, 1, 1, 1, 128), (1, 8, 16, 40, 256), (2, 2, 4, 17, 128), (5, 3, 8, 130, 640), (9, 1, 1, 64, 1024), (40, 4, 8, 96, 384),
    (33, 2, 5, 250, 1152), (7, 7, 1000, 16, 128), (70, 8, 9, 34, 2048), (3, 2, 3, 700, 256), (300, 2, 3, 66, 512), (64, 8, 64, 24, 128),
]


@pytest.mark.parametrize("T,k,E,N,K", SHAPES)
@pytest.mark.parametrize("gated", [False, True])
def test_experts(T, k, E, N, K, gated):
    if gated and N % 2:
        N += 1
    check_experts(T, k, E, N, K, gated, seed=1)
    check_experts(T, k, E, N, K, gated, pairs=True, pad=8, seed=2, globals_=False)


def test_experts_one_expert_has_all_and_none():
    for e, E in ((0, 3), (2, 3), (-1, 3), (700, 1024)):
        ids = torch.full((45, 2), e, dtype=torch.int32, device=DEV)
        check_experts(45, 2, E, 32, 256, False, ids=ids)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("counts", [[700, 0, 3, 193, 0, 1], [192, 384, 385, 0], [1, 1, 1, 1], [0, 0, 0, 4000]])
def test_experts_of_all_sizes_in_one_call(counts, gated):
    """Tiles of pairs of every width, several to an expert, empty experts between, and an odd number of 128 K."""
    ids = torch.cat([torch.full((n,), e, dtype=torch.int32) for e, n in enumerate(counts)])
    ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(1))].to(DEV).view(-1, 1)
    check_experts(len(ids), 1, len(counts), 300, 640, gated, seed=3, ids=ids)


@pytest.mark.parametrize("T,K", [(3, 256), (200, 384)])
def test_experts_same_expert_twice(T, K):
    """Two slots of a token may name one expert: two pairs with equal rows."""
    ids = torch.randint(0, 3, (T, 1), generator=gen(T), device=DEV, dtype=torch.int32).repeat(1, 2)
    w, s, gs = make_experts(3, 50, K, 6)
    a = torch.randn((T, K), generator=gen(7), device=DEV).bfloat16()
    got = wqp.w4a16_experts(a, w, s, *wqp.expert_order(ids, 3), 50, K, gs).view(T, 2, 50)
    assert torch.equal(got[:, 0], got[:, 1])


@pytest.mark.parametrize("T", [5, 400])
def test_experts_other_rows_and_offsets(T):
    """Positions that name no pair are passed over, offsets that go back or out of range are taken as far as they go:
    nothing outside the tensors is read or written."""
    E, k, N, K = 6, 2, 40, 256
    w, s, gs = make_experts(E, N, K, 8)
    a = torch.randn((T, K), generator=gen(9), device=DEV).bfloat16()
    ids = torch.randint(0, E, (T, k), generator=gen(10), device=DEV, dtype=torch.int32)
    rows, offsets = wqp.expert_order(ids, E)
    clean = wqp.w4a16_experts(a, w, s, rows, offsets, N, K, gs)
    bad = rows.clone()
    bad[::3] = torch.tensor([-1, -2 ** 31, 2 ** 31 - 1, T * k], device=DEV, dtype=torch.int32).repeat(T)[:len(bad[::3])]
    out = torch.full_like(clean, -5.0)
    wqp.w4a16_experts(a, w, s, bad, offsets, N, K, gs, out=out)
    hit = torch.zeros(T * k, dtype=torch.bool, device=DEV)
    hit[rows[::3].long()] = True
    assert (out[hit] == -5).all() and torch.equal(out[~hit], clean[~hit])
    for values in ([0, 4, 2, 8, 3, 9, 10], [-7, 2 ** 31 - 1, 0, -2 ** 31, 5, 5, 1], [2 ** 31 - 1] * 7, [-1] * 7):
        out.fill_(-5.0)
        wqp.w4a16_experts(a, w, s, rows, torch.tensor(values, device=DEV, dtype=torch.int32), N, K, gs, out=out)
        assert out.isfinite().all()


@pytest.mark.parametrize("gated", [False, True])
def test_experts_long_k(gated):
    check_experts(3, 2, 2, 20, 65536, gated, seed=9)
    check_experts(40, 2, 2, 20, 32768 + 128, gated, seed=9)


@pytest.mark.parametrize("T", [2, 200])
def test_experts_exact_integers(T):
    """Small whole activations, scales of 1: every partial sum is a multiple of 1/2 below 2^23."""
    E, k, N, K = 4, 2, 80, 512
    g = gen(11)
    w = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.full((E, N, K // 16), 0x38, device=DEV, dtype=torch.uint8)
    a = torch.randint(-4, 5, (T, K), generator=g, device=DEV).bfloat16()
    ids = torch.randint(0, E, (T, k), generator=g, device=DEV, dtype=torch.int32)
    got = wqp.w4a16_experts(a, w, s, *wqp.expert_order(ids, E), N, K)
    want, _, _ = experts64(a, w, s, None, ids, False, k)
    assert torch.equal(got.cpu(), want.float().bfloat16())


@pytest.mark.parametrize("T", [4, 200])
def test_experts_rows_do_not_touch_each_other(T):
    """Rows of infinities and NaNs, weights' NaN scales: only their own outputs show it; magnitudes of 2^+-40."""
    E, k, N, K = 3, 2, 48, 384
    g = gen(12)
    w, s, gs = make_experts(E, N, K, 4)
    a = torch.randn((T, K), generator=g, device=DEV).bfloat16()
    ids = torch.randint(0, E, (T, k), generator=g, device=DEV, dtype=torch.int32)
    order = wqp.expert_order(ids, E)
    clean = wqp.w4a16_experts(a, w, s, *order, N, K, gs)
    bad = a.clone()
    bad[1, 200] = NAN
    bad[3, 5] = INF
    got = wqp.w4a16_experts(bad, w, s, *order, N, K, gs)
    keep = torch.ones(T * k, dtype=torch.bool, device=DEV)
    keep[2:4] = keep[6:8] = False
    assert torch.equal(got[keep], clean[keep]) and got[2:4].isnan().all() and not got[6:8].isfinite().any()
    s2 = s.clone()
    s2[1, 7, 3] = 0x7F
    got = wqp.w4a16_experts(a, w, s2, *order, N, K, gs)
    hit = (ids.view(-1) == 1)
    assert got[hit][:, 7].isnan().all()
    got[hit, 7] = clean[hit, 7]
    assert torch.equal(got, clean)
    for e in (-40, 40):
        assert torch.equal(wqp.w4a16_experts(a * 2.0 ** e, w, s, *order, N, K, gs).float() * 2.0 ** -e, clean.float())


@pytest.mark.parametrize("T", [2, 60])
@pytest.mark.parametrize("gated", [False, True])
def test_experts_small_rows_with_small_global_scales(T, gated):
    """Outputs in BF16's range from rows and global scales whose powers of two alone FP32 does not hold; none from no weights."""
    E, k, N, K = 2, 2, 48, 512
    g = gen(14)
    w = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.full((E, N, K // 16), 0x7E, dtype=torch.uint8, device=DEV)
    a = torch.randn((T, K), generator=g, device=DEV)
    ids = torch.randint(0, E, (T, k), generator=g, device=DEV, dtype=torch.int32)
    order = wqp.expert_order(ids, E)
    for rows, globals_ in ((2.0 ** -86, 2.0 ** -48), (2.0 ** -16, 2.0 ** -120)):
        small = (a * rows).bfloat16()
        gs = torch.tensor([1.37, 0.71], device=DEV) * globals_
        if gated:
            gs = gs * 2.0 ** (58 if rows < 2.0 ** -80 else 60)
        got = wqp.w4a16_experts(small, w, s, *order, N, K, gs, gated).double().cpu()
        want, tol, _ = experts64(small, w, s, gs, ids, gated, k)
        assert ((got - want).abs() <= tol).all()
    large = (a * 2.0 ** 100).bfloat16()
    got = wqp.w4a16_experts(large, torch.zeros_like(w), s, *order, N, K, torch.full((E,), 2.0 ** 50, device=DEV), gated)
    assert (got == 0).all()


def test_experts_pairs_across_the_end_of_a_large_buffer():
    """Weights and outputs beyond 2^31 elements from their base."""
    E, N, K = 220, 4096, 5120
    g = gen(13)
    w = torch.zeros((E, N, K // 2), dtype=torch.uint8, device=DEV)
    s = torch.zeros((E, N, K // 16), dtype=torch.uint8, device=DEV)
    w[-1] = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    s[-1] = 0x30
    a = torch.randn((3, K), generator=g, device=DEV).bfloat16()
    ids = torch.tensor([[E - 1], [0], [E - 1]], dtype=torch.int32, device=DEV)
    got = wqp.w4a16_experts(a, w, s, *wqp.expert_order(ids, E), N, K).double().cpu()
    want, tol, _ = experts64(a[[0, 2]], w[-1:], s[-1:], None, torch.zeros(2, 1, dtype=torch.int32), False, 1)
    assert ((got[[0, 2]] - want).abs() <= tol).all() and (got[1] == 0).all()


# ---------------------------------------------------------------- combining
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,H,pad", [(1, 1, 8, 0), (1, 8, 5120, 0), (3, 2, 24, 8), (17, 32, 136, 16), (40, 5, 1000, 0), (257, 8, 128, 40), (9, 9, 65536, 0)])
@pytest.mark.parametrize("with_residual", [False, True])
def test_combine(dtype, T, k, H, pad, with_residual):
    g, E = gen(T + H), 11
    buf = torch.full((T * k, H + pad), 3.0, dtype=dtype, device=DEV)
    y = buf[:, :H]
    y.copy_(torch.randn((T * k, H), generator=g, device=DEV))
    ids = torch.randint(-2, E + 2, (T, k), generator=g, device=DEV, dtype=torch.int32)
    ids[0] = -1                                              # a token without any
    dead = (ids < 0) | (ids >= E)
    y[dead.view(-1)] = NAN
    weights = torch.rand((T, k), generator=g, device=DEV)
    weights[dead] = NAN
    res = torch.randn((T, H + pad), generator=g, device=DEV).to(dtype)[:, :H] if with_residual else None
    canvas = torch.full((T, H + pad), -5.0, dtype=dtype, device=DEV)
    out = wqp.expert_combine(y, weights, ids, E, residual=res, out=canvas[:, :H])
    w = torch.where(dead, 0.0, weights.double()).cpu().unsqueeze(2)
    v = torch.where(dead.view(-1, 1), 0.0, y.double()).cpu().view(T, k, H)
    want, S = (w * v).sum(1), (w * v).abs().sum(1)
    if with_residual:
        want, S = want + res.double().cpu(), S + res.double().cpu().abs()
    half = torch.finfo(dtype).eps / 2
    assert ((out.double().cpu() - want).abs() <= 35 * U * S * (1 + half) + half * want.abs() + 2.0 ** -25 * (dtype is torch.float16)).all()
    assert (canvas[:, H:] == -5).all()
    if with_residual:
        same = res.clone() if not pad else None
        if same is not None:
            assert wqp.expert_combine(y, weights, ids, E, residual=same, out=same).data_ptr() == same.data_ptr()
            assert torch.equal(same, out)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,H", [(1, 3, 16), (23, 9, 160), (300, 2, 2080)])
def test_combine_same_bits_whatever_the_alignment(dtype, T, k, H):
    """Bases and pitches of 32 bytes, and of 16: each in turn, and all."""
    g, E, step = gen(T + k), 5, 128 // torch.finfo(dtype).bits
    ids = torch.randint(-1, E, (T, k), generator=g, device=DEV, dtype=torch.int32)
    weights = torch.rand((T, k), generator=g, device=DEV)
    y, res = torch.randn((T * k, H), generator=g, device=DEV).to(dtype), torch.randn((T, H), generator=g, device=DEV).to(dtype)

    def place(x, base, pitch):
        buf = torch.full((x.shape[0] + 1, H + 16), 7.0, dtype=dtype, device=DEV).view(-1)
        return buf.as_strided(x.shape, (H + pitch * 8, 1), base * step).copy_(x)

    want = wqp.expert_combine(y, weights, ids, E, residual=res)
    for how in ((0, 0, 0, 0, 0, 0), (1, 0, 0, 0, 0, 0), (0, 1, 0, 0, 0, 0), (0, 0, 1, 0, 0, 0), (0, 0, 0, 1, 0, 0), (0, 0, 0, 0, 1, 0),
                (0, 0, 0, 0, 0, 1), (1, 1, 1, 1, 1, 1), (0, 2, 0, 2, 0, 2)):
        out = place(torch.zeros_like(res), *how[4:])
        got = wqp.expert_combine(place(y, *how[:2]), weights, ids, E, residual=place(res, *how[2:4]), out=out)
        assert torch.equal(got, want)


# ---------------------------------------------------------------- together
class Block:
    """A feed-forward part of E experts."""

    def __init__(self, H, F, E, k, seed=0):
        self.H, self.F, self.E, self.k = H, F, E, k
        self.up, self.down = make_experts(E, 2 * F, H, seed), make_experts(E, H, F, seed + 1)
        g = gen(seed + 2)
        self.router = torch.randn((H, E), generator=g, device=DEV) * H ** -0.5
        self.bias = torch.randn(E, generator=g, device=DEV) * 0.05

    def __call__(self, x, residual):
        ids, weights = wqp.expert_route(x.float() @ self.router, self.k, "sigmoid", self.bias, 4, 2)
        rows, offsets = wqp.expert_order(ids, self.E)
        u = wqp.w4a16_experts(x, self.up[0], self.up[1], rows, offsets, 2 * self.F, self.H, self.up[2], gated=True)
        y = wqp.w4a16_experts(u, self.down[0], self.down[1], rows, offsets, self.H, self.F, self.down[2])
        return ids, weights, u, y, wqp.expert_combine(y, weights, ids, self.E, residual=residual)


@pytest.mark.parametrize("T", [1, 19, 260])
def test_block(T):
    """Each step against its 64-bit form on what the step before gave."""
    b = Block(512, 256, 16, 4)
    g = gen(T)
    x, r = (torch.randn((T, b.H), generator=g, device=DEV).bfloat16() for _ in range(2))
    ids, weights, u, y, out = b(x, r)
    want, tol, _ = experts64(x, b.up[0], b.up[1], b.up[2], ids, True, b.k)
    assert ((u.double().cpu() - want).abs() <= tol).all()
    want, tol, _ = experts64(u, b.down[0], b.down[1], b.down[2], ids, False, 1)
    assert ((y.double().cpu() - want).abs() <= tol).all()
    v = weights.double().cpu().unsqueeze(2) * y.double().cpu().view(T, b.k, b.H)
    want = v.sum(1) + r.double().cpu()
    assert ((out.double().cpu() - want).abs() <= 35 * U * (v.abs().sum(1) + r.double().cpu().abs()) * 1.01 + 2.0 ** -8 * want.abs()).all()


@pytest.mark.parametrize("T", [1, 6, 300])
@pytest.mark.parametrize("pdl", [False, True])
def test_block_in_a_graph(T, pdl):
    """Captured once and replayed for other tokens, which choose other experts; under programmatic dependent launch too."""
    b = Block(512, 256, 16, 4)
    g = gen(100 + T)
    inputs = [[torch.randn((T, b.H), generator=g, device=DEV).bfloat16() for _ in range(2)] for _ in range(5)]
    want = [[t.clone() for t in b(*i)] for i in inputs]
    x, r = (t.clone() for t in inputs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b(x, r)
    torch.cuda.current_stream().wait_stream(side)
    old = wqp.set_pdl(pdl)
    try:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = b(x, r)
        for _ in range(3):
            for i, w in zip(inputs, want):
                x.copy_(i[0])
                r.copy_(i[1])
                graph.replay()
                assert all(torch.equal(p, q) for p, q in zip(got, w))
    finally:
        wqp.set_pdl(old)


@pytest.mark.parametrize("T", [1, 300])
def test_block_under_programmatic_dependent_launch(T):
    """Call after call into the same buffers with other tokens each time: a value left from before would show."""
    b = Block(512, 256, 16, 4)
    g = gen(150 + T)
    inputs = [[torch.randn((T, b.H), generator=g, device=DEV).bfloat16() for _ in range(2)] for _ in range(4)]
    logits = [i[0].float() @ b.router for i in inputs]
    order = (torch.empty(T * 4, dtype=torch.int32, device=DEV), torch.empty(17, dtype=torch.int32, device=DEV))
    routed = (torch.empty((T, 4), dtype=torch.int32, device=DEV), torch.empty((T, 4), device=DEV))
    u, y, out = (torch.empty((n, m), dtype=torch.bfloat16, device=DEV) for n, m in ((T * 4, 256), (T * 4, 512), (T, 512)))

    def chain(i):
        wqp.expert_route(logits[i], 4, "sigmoid", b.bias, 4, 2, out=routed)
        wqp.expert_order(routed[0], 16, out=order)
        wqp.w4a16_experts(inputs[i][0], b.up[0], b.up[1], *order, 512, 512, b.up[2], gated=True, out=u)
        wqp.w4a16_experts(u, b.down[0], b.down[1], *order, 512, 256, b.down[2], out=y)
        wqp.expert_combine(y, routed[1], routed[0], 16, residual=inputs[i][1], out=out)
        return [*routed, *order, u, y, out]

    want = [[t.clone() for t in chain(i)] for i in range(4)]
    torch.cuda.synchronize()
    old = wqp.set_pdl(True)
    try:
        for _ in range(4):
            for i in range(4):
                got = [t.clone() for t in chain(i)]
                assert all(torch.equal(p, q) for p, q in zip(got, want[i]))
    finally:
        wqp.set_pdl(old)


@pytest.mark.parametrize("T", [1, 300])
def test_block_on_other_streams(T):
    b = Block(512, 256, 16, 4)
    g = gen(200 + T)
    x, r = (torch.randn((T, b.H), generator=g, device=DEV).bfloat16() for _ in range(2))
    want = [t.clone() for t in b(x, r)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams * 2:
        with torch.cuda.stream(s):
            got.append(b(x, r))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for many in got for p, q in zip(many, want))
    # The stream as an argument.
    s = streams[0]
    ids, weights = wqp.expert_route(x.float() @ b.router, 4, "sigmoid", b.bias, 4, 2, stream=torch.cuda.current_stream())
    s.wait_stream(torch.cuda.current_stream())
    rows, offsets = wqp.expert_order(ids, b.E, stream=s)
    u = wqp.w4a16_experts(x, b.up[0], b.up[1], rows, offsets, 2 * b.F, b.H, b.up[2], gated=True, stream=s)
    y = wqp.w4a16_experts(u, b.down[0], b.down[1], rows, offsets, b.H, b.F, b.down[2], stream=s)
    out = wqp.expert_combine(y, weights, ids, b.E, residual=r, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(p, q) for p, q in zip((ids, weights, u, y, out), want))
