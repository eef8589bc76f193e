"""The mixture-of-experts operators of the packed-weight path, measured.

Four operators: expert_route (scores of a token's experts to its top_k experts and their weights), expert_order (the
(token, slot) pairs grouped by expert), w4a16_experts (each pair's row times its expert's packed W4A16 matrix, plain or as
silu(gate) * up) and expert_combine (a token's rows, weighted and added).

A pass is one call on the inputs that prepare() makes. Where `own` is false it runs the plain form, in torch operations in
FP32 (the order of the experts in FP64: two scores may lie closer than FP32 tells apart); where it is true, the
framework's entry points. A pair that has no expert (id -1: padding, or an expert kept elsewhere) is not computed.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    grouped = {"E": 256, "top_k": 8, "scoring": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "group_best": 2,
               "renormalise": True, "scale": 2.5, "type": "f32", "masked": False}
    plain = {"E": 128, "top_k": 8, "scoring": "softmax", "bias": False, "groups": 1, "top_groups": 1, "group_best": 2,
             "renormalise": True, "scale": 1.0, "type": "bf16", "masked": False}
    return [
        # One token's routing, by groups with a balancing bias; then a long prompt's, an odd number of tokens, and by softmax.
        {"name": "expert_route 1x256 groups", "op": "expert_route", "T": 1, "pad": 0, **grouped},
        {"name": "expert_route 8191x256 groups", "op": "expert_route", "T": 8191, "pad": 0, **grouped},
        {"name": "expert_route 8192x128 softmax", "op": "expert_route", "T": 8192, "pad": 0, **plain},
        # The pairs of one token, and of a long prompt.
        {"name": "expert_order 1x8 of 256", "op": "expert_order", "T": 1, "top_k": 8, "E": 256, "dropped": 0.0},
        {"name": "expert_order 8192x8 of 256", "op": "expert_order", "T": 8192, "top_k": 8, "E": 256, "dropped": 0.0},
        # Gate and up for one token; down for a decode batch; gate and up for a short odd prompt; both for a long one.
        {"name": "w4a16_experts 1x8 of 128, gated 4096x5120", "op": "w4a16_experts", "T": 1, "top_k": 8, "E": 128, "N": 4096, "K": 5120,
         "gated": True, "pairs": False, "pad": 0, "dropped": 0.0, "skew": 0.0},
        {"name": "w4a16_experts 16x8 of 128, 5120x2048", "op": "w4a16_experts", "T": 16, "top_k": 8, "E": 128, "N": 5120, "K": 2048,
         "gated": False, "pairs": True, "pad": 0, "dropped": 0.0, "skew": 0.0},
        {"name": "w4a16_experts 333x8 of 128, gated 4096x5120", "op": "w4a16_experts", "T": 333, "top_k": 8, "E": 128, "N": 4096, "K": 5120,
         "gated": True, "pairs": False, "pad": 0, "dropped": 0.0, "skew": 0.0},
        {"name": "w4a16_experts 4096x8 of 128, gated 4096x5120", "op": "w4a16_experts", "T": 4096, "top_k": 8, "E": 128, "N": 4096, "K": 5120,
         "gated": True, "pairs": False, "pad": 0, "dropped": 0.0, "skew": 0.0},
        {"name": "w4a16_experts 4096x8 of 128, 5120x2048", "op": "w4a16_experts", "T": 4096, "top_k": 8, "E": 128, "N": 5120, "K": 2048,
         "gated": False, "pairs": True, "pad": 0, "dropped": 0.0, "skew": 0.0},
        # The sum of one token's rows; of a long prompt's, with the residual.
        {"name": "expert_combine 1x8x5120", "op": "expert_combine", "T": 1, "top_k": 8, "H": 5120, "E": 128, "type": "bf16", "pad": 0,
         "residual": True, "dropped": 0.0},
        {"name": "expert_combine 8192x8x5120", "op": "expert_combine", "T": 8192, "top_k": 8, "H": 5120, "E": 128, "type": "bf16", "pad": 0,
         "residual": True, "dropped": 0.0},
    ]


def _spread(rng, lo, hi, unit=1):
    """A multiple of `unit` between lo and hi, spread over the logarithm."""
    return unit * max(1, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))) // unit)


def draw(rng):
    op = rng.choice(["expert_route", "expert_order", "w4a16_experts", "w4a16_experts", "w4a16_experts", "expert_combine"])
    c = {"op": op, "T": _spread(rng, 1, 8192)}
    if op == "expert_route":
        groups = rng.choice([1, 1, 2, 4, 8])
        c["T"] = _spread(rng, 4, 8192)
        c["E"] = groups * _spread(rng, 8, 1024 // groups)
        c["groups"], c["top_groups"] = groups, rng.randint(1, groups)
        c["group_best"] = rng.choice([1, 2])
        c["top_k"] = rng.randint(1, min(16, c["E"] // groups * c["top_groups"]))
        c["scoring"] = rng.choice(["softmax", "sigmoid"])
        c["bias"], c["renormalise"], c["masked"] = rng.random() < 0.5, rng.random() < 0.7, rng.random() < 0.3
        c["scale"] = rng.choice([1.0, 2.5])
        c["type"] = rng.choice(["bf16", "f16", "f32"])
        c["pad"] = rng.choice([0, 0, 3, 8])
        return c
    c["E"] = _spread(rng, 1, 256)
    c["top_k"] = rng.randint(1, min(8, c["E"]))
    c["dropped"] = rng.choice([0.0, 0.0, 0.3])
    if op == "expert_order":
        c["T"], c["E"], c["top_k"] = _spread(rng, 4, 8192), _spread(rng, 16, 1024), rng.randint(2, 8)
    if op == "expert_combine":
        c["H"] = _spread(rng, 128, 8192, 8)
        c["type"] = rng.choice(["bf16", "bf16", "f16", "f32"])
        c["pad"] = rng.choice([0, 0, 8, 40])
        c["residual"] = rng.random() < 0.5
        c["T"] = _spread(rng, 1, max(1, min(8192, 8192 * 8 * 5120 // (c["top_k"] * c["H"] * (2 if c["type"] == "f32" else 1)))))
    if op == "w4a16_experts":
        c["K"] = _spread(rng, 128, 8192, 128)
        c["gated"] = rng.random() < 0.5
        most = max(2, min(8192, 128 * 4096 * 5120 // (c["E"] * c["K"])))
        c["N"] = 2 * _spread(rng, 1, most // 2) if c["gated"] else _spread(rng, 1, most)
        c["T"] = _spread(rng, 1, max(1, min(4096, 4096 * 8 * 4096 * 5120 // (c["top_k"] * c["N"] * c["K"]))))
        c["pairs"] = not c["gated"]
        c["pad"] = rng.choice([0, 0, 8, 40])
        c["skew"] = rng.choice([0.0, 1.0])
    return c


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _padded(rows, cols, pad, dtype):
    """An uninitialised [rows, cols] tensor whose rows are cols + pad apart."""
    return torch.empty((rows, cols + pad), dtype=dtype, device=DEV)[:, :cols]


def _ids(case, gen):
    """top_k different experts a token, the skewed ones some far more often than others; a share of the pairs dropped."""
    T, E, k = case["T"], case["E"], case["top_k"]
    scores = torch.rand((T, E), generator=gen, device=DEV) + case.get("skew", 0.0) * torch.randn(E, generator=gen, device=DEV)
    ids = torch.topk(scores, k, dim=1).indices.to(torch.int32)
    if case["dropped"]:
        ids[torch.rand((T, k), generator=gen, device=DEV) < case["dropped"]] = -1
    return ids


def _ordered(ids, E):
    """Pairs by expert, in their own order within one, -1 behind the last; and where each expert's begin."""
    flat = ids.view(-1)
    live = (flat >= 0) & (flat < E)
    key = torch.where(live, flat, E)
    rows = torch.sort(key, stable=True).indices.to(torch.int32)
    count = (key.unsqueeze(0) == torch.arange(E, device=DEV).unsqueeze(1)).sum(1)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(count, 0)
    rows[torch.arange(flat.numel(), device=DEV) >= offsets[E]] = -1
    return rows, offsets


# ------------------------------------------------------------------ plain forms
def _route(st, weight_type):
    """ids and weights: the order in FP64, the weights in weight_type."""
    c, E, k = st["case"], st["case"]["E"], st["case"]["top_k"]
    x = st["logits"].double()
    live = x > float("-inf")
    top = torch.where(live, x, -1e300).amax(1, keepdim=True)
    if c["scoring"] == "softmax":
        e = torch.where(live, torch.exp(x - top), 0.0)
        s = e / e.sum(1, keepdim=True).clamp_min(1e-300)
    else:
        s = torch.where(live, 1.0 / (1.0 + torch.exp(-x)), 0.0)
    choice = torch.where(live, s + st["bias"].double(), float("-inf")) if st["bias"] is not None else x
    if c["groups"] > 1:
        by_group = (s + st["bias"].double() if st["bias"] is not None else (s if c["group_best"] == 2 else x)).view(-1, c["groups"], E // c["groups"])
        alive = live.view(by_group.shape)
        best = torch.where(alive, by_group, float("-inf")).sort(2, descending=True).values[:, :, :c["group_best"]]
        score = torch.where(best > float("-inf"), best, 0.0).sum(2)
        score = torch.where(alive.any(2), score, float("-inf"))
        order = torch.sort(score, dim=1, descending=True, stable=True).indices
        chosen = torch.zeros_like(score, dtype=torch.bool).scatter_(1, order[:, :c["top_groups"]], True)
        choice = torch.where(chosen.repeat_interleave(E // c["groups"], 1), choice, float("-inf"))
    values, order = torch.sort(choice, dim=1, descending=True, stable=True)
    found = values[:, :k] > float("-inf")
    ids = torch.where(found, order[:, :k], -1).to(torch.int32)
    w = torch.where(found, s.gather(1, order[:, :k]), 0.0).to(weight_type)
    if c["renormalise"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / torch.where(total > 0, total, 1.0), 0.0)
    return {"ids": ids, "weights": w * c["scale"]}


def _expert_weights(st, e, real):
    """Expert e's matrix without its global scale."""
    codes, scales = st["w"][e], st["w_scales"][e].view(torch.float8_e4m3fn).to(real)
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=real, device=DEV)
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), 2).view(codes.shape[0], -1, 16)
    return (v * scales.unsqueeze(2)).view(codes.shape[0], -1)


def _experts(st, real):
    c = st["case"]
    flat = st["ids"].view(-1)
    F = c["N"] // 2 if c["gated"] else c["N"]
    out = torch.zeros((flat.numel(), F), dtype=real, device=DEV)
    for e in torch.unique(flat[flat >= 0]).tolist():
        at = (flat == e).nonzero().view(-1)
        a = st["a"][at if c["pairs"] else at // c["top_k"]].to(real)
        u = (a @ _expert_weights(st, e, real).t()) * st["globals"][e].to(real)
        out[at] = u[:, :F] / (1.0 + torch.exp(-u[:, :F])) * u[:, F:] if c["gated"] else u
    return out


def _combine(st, real):
    T, k, H = st["case"]["T"], st["case"]["top_k"], st["case"]["H"]
    live = (st["ids"] >= 0).unsqueeze(2)
    got = torch.zeros((T, H), dtype=real, device=DEV)
    for s in range(k):
        row = st["y"][s::k].to(real) * st["weights"][:, s:s + 1].to(real)
        got += torch.where(live[:, s], row, 0.0)
    return got if st["residual"] is None else got + st["residual"].to(real)


def _plain(st):
    c = st["case"]
    if c["op"] == "expert_route":
        return _route(st, torch.float32)
    if c["op"] == "expert_order":
        rows, offsets = _ordered(st["ids"], c["E"])
        return {"rows": rows, "offsets": offsets}
    if c["op"] == "w4a16_experts":
        return _experts(st, torch.float32).to(torch.bfloat16)
    return _combine(st, torch.float32).to(st["y"].dtype)


# ------------------------------------------------------------------ the framework's
def _own(st):
    import weight_only_quantized_packed_gb300 as wqp

    c = st["case"]
    if c["op"] == "expert_route":
        ids, weights = wqp.expert_route(st["logits"], c["top_k"], scoring=c["scoring"], bias=st["bias"], groups=c["groups"],
                                        top_groups=c["top_groups"], group_best=c["group_best"], renormalise=c["renormalise"],
                                        scale=c["scale"], out=st["out"])
        return {"ids": ids, "weights": weights}
    if c["op"] == "expert_order":
        rows, offsets = wqp.expert_order(st["ids"], c["E"], out=st["out"])
        return {"rows": rows, "offsets": offsets}
    if c["op"] == "w4a16_experts":
        return wqp.w4a16_experts(st["a"], st["w"], st["w_scales"], st["rows"], st["offsets"], c["N"], c["K"], st["globals"],
                                 gated=c["gated"], out=st["out"])
    return wqp.expert_combine(st["y"], st["weights"], st["ids"], c["E"], residual=st["residual"], out=st["out"])


def prepare(case, seed):
    gen = _gen(seed)
    op, T, E, k = case["op"], case["T"], case["E"], case["top_k"]
    st = {"case": case}
    if op == "expert_route":
        st["logits"] = _padded(T, E, case["pad"], TYPES[case["type"]])
        st["logits"].copy_(2.0 * torch.randn((T, E), generator=gen, device=DEV))
        if case["masked"]:                       # experts that may not be used, and rows that may use none
            st["logits"][torch.rand((T, E), generator=gen, device=DEV) < 0.5] = float("-inf")
            st["logits"][torch.rand(T, generator=gen, device=DEV) < 0.05] = float("-inf")
        st["bias"] = 0.1 * torch.randn(E, generator=gen, device=DEV) if case["bias"] else None
        st["out"] = (torch.empty((T, k), dtype=torch.int32, device=DEV), torch.empty((T, k), device=DEV))
        return st
    st["ids"] = _ids(case, gen)
    if op == "expert_order":
        st["out"] = (torch.empty(T * k, dtype=torch.int32, device=DEV), torch.empty(E + 1, dtype=torch.int32, device=DEV))
    elif op == "w4a16_experts":
        N, K = case["N"], case["K"]
        st["rows"], st["offsets"] = _ordered(st["ids"], E)
        st["a"] = _padded(T * k if case["pairs"] else T, K, case["pad"], torch.bfloat16)
        # Hidden-state-like rows: normal values, and one channel in 64 sixteen times as large.
        st["a"].copy_(torch.randn(st["a"].shape, generator=gen, device=DEV))
        st["a"] *= torch.where(torch.rand(K, generator=gen, device=DEV) < 1 / 64, 16.0, 1.0).bfloat16()
        # Weights as the packed format's own recipe draws them: every nibble, half-normal scales.
        st["w"] = torch.randint(0, 256, (E, N, K // 2), generator=gen, device=DEV, dtype=torch.uint8)
        scales = torch.empty((E, N, K // 16), dtype=torch.float8_e4m3fn, device=DEV)
        for e in range(E):
            scales[e] = (torch.randn((N, K // 16), generator=gen, device=DEV).abs() * 0.05).to(torch.float8_e4m3fn)
        st["w_scales"] = scales.view(torch.uint8)
        st["globals"] = (0.5 + torch.rand(E, generator=gen, device=DEV)) * (0.25 if case["gated"] else 1.0)
        st["out"] = torch.zeros((T * k, (N // 2 if case["gated"] else N) + case["pad"]), dtype=torch.bfloat16, device=DEV)[:, :N // 2 if case["gated"] else N]
    else:
        H, dtype = case["H"], TYPES[case["type"]]
        st["y"] = _padded(T * k, H, case["pad"], dtype)
        st["y"].copy_(torch.randn((T * k, H), generator=gen, device=DEV))
        st["y"][st["ids"].view(-1) < 0] = float("nan")        # what was never computed
        st["weights"] = torch.softmax(torch.randn((T, k), generator=gen, device=DEV), 1)
        st["residual"] = None
        if case["residual"]:
            st["residual"] = _padded(T, H, case["pad"], dtype)
            st["residual"].copy_(4.0 * torch.randn((T, H), generator=gen, device=DEV))
        st["out"] = torch.empty((T, H), dtype=dtype, device=DEV)
    return st


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op, T, E, k = case["op"], case["T"], case["E"], case["top_k"]
    if op == "expert_route":
        size = {"bf16": 2, "f16": 2, "f32": 4}[case["type"]]
        return {"bytes": T * E * size + (4 * E if case["bias"] else 0) + 8 * T * k, "flops": 4 * T * E}
    if op == "expert_order":
        return {"bytes": 8 * T * k + 4 * (E + 1), "flops": T * k}
    kept = 1.0 - case["dropped"]
    pairs = T * k * kept
    if op == "w4a16_experts":
        N, K = case["N"], case["K"]
        used = E * (1.0 - (1.0 - k * kept / E) ** T)          # experts that some token chose, on average
        rows = pairs if case["pairs"] else T
        width = N // 2 if case["gated"] else N
        return {"bytes": used * N * K * 9 / 16 + 2 * rows * K + 2 * pairs * width + 4 * (T * k + 2 * E), "flops": 2 * pairs * N * K}
    size = {"bf16": 2, "f16": 2, "f32": 4}[case["type"]]
    return {"bytes": case["H"] * size * (pairs + T * (2 if case["residual"] else 1)) + 8 * T * k, "flops": 2 * pairs * case["H"]}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op, T, E, k = case["op"], case["T"], case["E"], case["top_k"]
    if op == "expert_order":
        flat = st["ids"].view(-1).tolist()
        rows, offsets = [], [0]
        lists = [[] for _ in range(E)]
        for i, e in enumerate(flat):
            if 0 <= e < E:
                lists[e].append(i)
        for at in lists:
            rows += at
            offsets.append(len(rows))
        rows += [-1] * (len(flat) - len(rows))
        return {"rows": torch.tensor(rows, dtype=torch.int32, device=DEV), "offsets": torch.tensor(offsets, dtype=torch.int32, device=DEV)}
    if op == "expert_route":
        x = st["logits"].double()
        p = torch.sigmoid(x) if case["scoring"] == "sigmoid" else torch.nan_to_num(torch.softmax(x, 1), nan=0.0)
        key = x.clone() if st["bias"] is None else torch.where(x == float("-inf"), x, p + st["bias"].double())
        if case["groups"] > 1:
            g = case["groups"]
            base = key if st["bias"] is not None or case["group_best"] == 1 else torch.where(x == float("-inf"), x, p)
            first = base.view(T, g, -1).amax(2)
            score = first
            if case["group_best"] == 2 and E // g > 1:
                second = base.view(T, g, -1).topk(2, dim=2).values[:, :, 1]
                score = torch.where(second == float("-inf"), first, first + second)
            for _ in range(g - case["top_groups"]):           # the worst group goes, of equal ones the last
                worst = g - 1 - torch.argmin(score.flip(1), 1)
                score[torch.arange(T, device=DEV), worst] = float("inf")
                key.view(T, g, -1)[torch.arange(T, device=DEV), worst] = float("-inf")
        ids = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
        w = torch.zeros((T, k), dtype=torch.float64, device=DEV)
        every = torch.arange(T, device=DEV)
        for s in range(k):                                    # the best of what is left, of equal ones the first
            best = key.amax(1)
            at = (key == best.unsqueeze(1)).int().argmax(1)
            ok = best > float("-inf")
            ids[:, s] = torch.where(ok, at, -1).int()
            w[:, s] = torch.where(ok, p[every, at], 0.0)
            key[every, at] = float("-inf")
        if case["renormalise"]:
            w = torch.nan_to_num(w / w.sum(1, keepdim=True), nan=0.0)
        return {"ids": ids, "weights": w * case["scale"]}
    if op == "w4a16_experts":
        F = case["N"] // 2 if case["gated"] else case["N"]
        out = torch.zeros((T * k, F), dtype=torch.float64, device=DEV)
        mags = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
        rows, offsets = st["rows"].long(), st["offsets"].tolist()
        for e in range(E):
            at = rows[offsets[e]:offsets[e + 1]]
            if not at.numel():
                continue
            w = torch.empty((case["N"], case["K"]), dtype=torch.float64, device=DEV)
            lo, hi = (st["w"][e] & 15).int(), (st["w"][e] >> 4).int()
            w[:, 0::2] = mags[lo & 7] * (1 - 2 * (lo >> 3))
            w[:, 1::2] = mags[hi & 7] * (1 - 2 * (hi >> 3))
            w *= st["w_scales"][e].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1) * st["globals"][e].double()
            u = st["a"][at if case["pairs"] else torch.div(at, k, rounding_mode="floor")].double() @ w.t()
            out[at] = u[:, :F] * torch.sigmoid(u[:, :F]) * u[:, F:] if case["gated"] else u
        return out
    w = torch.where(st["ids"] >= 0, st["weights"].double(), 0.0)
    y = torch.where((st["ids"] >= 0).view(-1, 1), st["y"].double(), 0.0).view(T, k, -1) if T * k * case["H"] <= 1 << 26 else None
    if y is not None:
        got = torch.einsum("tk,tkh->th", w, y)
    else:
        got = torch.empty((T, case["H"]), dtype=torch.float64, device=DEV)
        for t in range(0, T, 1024):
            part = st["y"][t * k:(t + 1024) * k].double().view(-1, k, case["H"])
            part = torch.where((st["ids"][t:t + 1024] >= 0).unsqueeze(2), part, 0.0)
            got[t:t + 1024] = torch.einsum("tk,tkh->th", w[t:t + 1024], part)
    return got if st["residual"] is None else got + st["residual"].double()
