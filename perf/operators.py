"""The quantised-activation operators of the packed-weight path, measured.

Five operators: w4_quantize (rows to E2M1 codes with an E4M3 scale per 16 and one FP32 scale), a8_quantize (rows to
E4M3 with an FP32 scale per 128), rms_norm with the residual's addition (its output in the inputs' type or as
a8_quantize writes it), w4a4_gemm and w8a8_gemm (products of such rows with packed weights of the same formats).

A pass is one call on the inputs that prepare() makes. Where `own` is false it runs the plain form, in FP32 torch
operations; where it is true, the framework's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
UNUSED = 3072                # no configuration of this repository has this size
FLOOR = 2.0 ** -100          # the least magnitude an 8-bit group's scale is taken from


def listed():
    return [
        # One token's activations on the way into a 4-bit projection; then a hidden-by-FFN weight matrix from FP32.
        {"name": "w4_quantize 1x5120", "op": "w4_quantize", "M": 1, "K": 5120, "type": "bf16", "pad": 0},
        {"name": "w4_quantize 17408x5120 f32", "op": "w4_quantize", "M": 17408, "K": 5120, "type": "f32", "pad": 0},
        # A decode batch's FFN activations; then a long prompt's, an odd number of rows.
        {"name": "a8_quantize 16x17408", "op": "a8_quantize", "M": 16, "K": 17408, "type": "bf16", "pad": 0},
        {"name": "a8_quantize 8191x17408", "op": "a8_quantize", "M": 8191, "K": 17408, "type": "bf16", "pad": 0},
        # The norm before a projection: one token, and a long prompt.
        {"name": "rms_norm_a8 1x5120", "op": "rms_norm", "M": 1, "K": 5120, "type": "bf16", "pad": 0, "out": "a8", "residual": True},
        {"name": "rms_norm_a8 8192x5120", "op": "rms_norm", "M": 8192, "K": 5120, "type": "bf16", "pad": 0, "out": "a8", "residual": True},
        # 4-bit products: one token through a square projection, a ragged mid batch through qkv, a prompt through gate+up.
        {"name": "w4a4_gemm 1x5120x5120", "op": "w4a4_gemm", "M": 1, "N": 5120, "K": 5120, "pad": 0},
        {"name": "w4a4_gemm 333x7168x5120", "op": "w4a4_gemm", "M": 333, "N": 7168, "K": 5120, "pad": 0},
        {"name": "w4a4_gemm 4096x34816x5120", "op": "w4a4_gemm", "M": 4096, "N": 34816, "K": 5120, "pad": 0},
        # 8-bit products: one token into the FFN, a small odd batch out of it, a prompt out of it.
        {"name": "w8a8_gemm 1x17408x5120", "op": "w8a8_gemm", "M": 1, "N": 17408, "K": 5120, "pad": 0},
        {"name": "w8a8_gemm 61x5120x17408", "op": "w8a8_gemm", "M": 61, "N": 5120, "K": 17408, "pad": 0},
        {"name": "w8a8_gemm 4096x5120x17408", "op": "w8a8_gemm", "M": 4096, "N": 5120, "K": 17408, "pad": 0},
    ]


def _spread(rng, lo, hi, unit=1):
    """A multiple of `unit` between lo and hi, spread over the logarithm; none is UNUSED."""
    v = unit * max(1, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))) // unit)
    return v if v != UNUSED else v - unit


def draw(rng):
    op = rng.choice(["w4_quantize", "a8_quantize", "rms_norm", "w4a4_gemm", "w8a8_gemm", "w4a4_gemm", "w8a8_gemm"])
    unit = 256 if op == "w4a4_gemm" else 128
    K = _spread(rng, 128, 17408, unit)
    c = {"op": op, "K": K, "pad": rng.choice([0, 0, 8, 40])}
    if op.endswith("gemm"):
        c["N"] = _spread(rng, 1, 34816)
        c["M"] = _spread(rng, 1, max(1, min(8192, 4096 * 34816 * 5120 // (c["N"] * K))))
    else:
        c["M"] = _spread(rng, 1, max(1, min(17408, 17408 * 5120 // K)))
        c["type"] = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "rms_norm":
        c["out"] = rng.choice(["a8", "same"])
        c["residual"] = rng.random() < 0.75
    return c


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _padded(rows, cols, pad, dtype):
    """An uninitialised [rows, cols] tensor whose rows are cols + pad apart."""
    return torch.empty((rows, cols + pad), dtype=dtype, device=DEV)[:, :cols]


def _activations(M, K, gen):
    """Hidden-state-like rows: normal values, and one channel in 64 sixteen times as large."""
    x = torch.randn((M, K), generator=gen, device=DEV)
    return x * torch.where(torch.rand(K, generator=gen, device=DEV) < 1 / 64, 16.0, 1.0)


def _bytes(*shape):
    return torch.empty(shape, dtype=torch.uint8, device=DEV)


# ------------------------------------------------------------------ plain forms (FP32)
def _e4m3(v):
    """Nearest E4M3 codes of v, saturating; NaN stays NaN."""
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _w4_codes(x, g):
    """x [M, K] FP32 -> codes 0..15 [M, K] uint8 and E4M3 scales [M, K/16]."""
    M, K = x.shape
    xg = x.view(M, K // 16, 16)
    g = torch.tensor(g, dtype=torch.float32, device=x.device)
    amax = xg.abs().amax(2)
    amax = torch.where(torch.isfinite(amax), amax, float("nan"))
    s = _e4m3(amax / (6.0 * g))
    d = (s.float() * g).unsqueeze(2)
    q = torch.where(d > 0, xg / d, 0.0)
    a = q.abs()
    mag = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return (mag | ((q < 0).to(torch.uint8) << 3)).view(M, K), s


def _pack4(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def _unpack4(packed):
    """Packed E2M1 bytes [R, K/2] -> FP32 values [R, K]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=packed.device)
    return torch.stack((table[(packed & 15).int()], table[(packed >> 4).int()]), 2).view(packed.shape[0], -1)


def _w4_values(packed, scales, g):
    v = _unpack4(packed)
    s = scales.view(torch.float8_e4m3fn).float()
    return ((v.view(s.shape[0], -1, 16) * s.unsqueeze(2)) * g).view(v.shape)


def _a8_codes(y):
    """y [M, K] FP32 -> E4M3 codes [M, K] and FP32 scales [M, K/128]."""
    M, K = y.shape
    yg = y.view(M, K // 128, 128)
    amax = yg.abs().amax(2).clamp_min(FLOOR)
    amax = torch.where(torch.isfinite(amax), amax, float("nan"))
    return _e4m3(yg * (448.0 / amax).unsqueeze(2)).view(M, K), amax / 448.0


def _plain(st):
    op = st["case"]["op"]
    if op == "w4_quantize":
        codes, s = _w4_codes(st["x"].float(), st["g"])
        return {"values": _w4_values(_pack4(codes), s.view(torch.uint8), st["g"]), "scales": s}
    if op == "a8_quantize":
        q, s = _a8_codes(st["x"].float())
        return {"codes": q, "scales": s}
    if op == "rms_norm":
        x, got = st["x"].float(), {}
        if st["residual"] is not None:
            x = x + st["residual"].float()
            got["residual"] = x.to(st["x"].dtype)
        y = x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * st["weight"].float()
        if st["case"]["out"] == "a8":
            got["codes"], got["scales"] = _a8_codes(y)
        else:
            got["y"] = y.to(st["x"].dtype)
        return got
    if op == "w4a4_gemm":
        a = _w4_values(st["a"], st["a_scales"], 1.0)
        w = _w4_values(st["w"], st["w_scales"], 1.0)
        return ((a @ w.t()) * (st["ga"] * st["gw"])).to(torch.bfloat16)
    a = (st["a"].view(torch.float8_e4m3fn).float().view(*st["a_scales"].shape, 128) * st["a_scales"].unsqueeze(2)).view(st["a"].shape)
    N, K = st["w"].shape
    s = st["w_scales"].repeat_interleave(128, 0)[:N].unsqueeze(2)
    w = (st["w"].view(torch.float8_e4m3fn).float().view(N, K // 128, 128) * s).view(N, K)
    return (a @ w.t()).to(torch.bfloat16)


# ------------------------------------------------------------------ the framework's
def _own(st):
    import weight_only_quantized_packed_gb300 as wqp

    op = st["case"]["op"]
    if op == "w4_quantize":
        codes, scales = wqp.w4_quantize(st["x"], st["g"], out=st["out"])
        M, K = st["x"].shape
        return {"values": wqp.w4a16_dequant(codes, scales, M, K, st["g"], out=st["values"]), "scales": scales.view(torch.float8_e4m3fn)}
    if op == "a8_quantize":
        codes, scales = wqp.a8_quantize(st["x"], out=st["out"])
        return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales}
    if op == "rms_norm":
        got = {}
        if st["case"]["out"] == "a8":
            codes, scales, h = wqp.rms_norm_a8(st["x"], st["weight"], EPS, residual=st["residual"], residual_out=st["residual_out"], out=st["out"])
            got["codes"], got["scales"] = codes.view(torch.float8_e4m3fn), scales
        else:
            got["y"], h = wqp.rms_norm(st["x"], st["weight"], EPS, residual=st["residual"], residual_out=st["residual_out"], out=st["out"])
        if st["residual"] is not None:
            got["residual"] = h
        return got
    N, K = st["case"]["N"], st["case"]["K"]
    if op == "w4a4_gemm":
        return wqp.w4a4_gemm(st["a"], st["a_scales"], st["w"], st["w_scales"], N, K, st["ga"], st["gw"], out=st["out"])
    return wqp.w8a8_gemm(st["a"], st["a_scales"], st["w"], st["w_scales"], N, K, out=st["out"])


def prepare(case, seed):
    gen = _gen(seed)
    op, M, K, pad = case["op"], case["M"], case["K"], case["pad"]
    st = {"case": case}
    if op.endswith("gemm"):
        N = case["N"]
        x = _activations(M, K, gen)
        st["out"] = _padded(M, N, pad, torch.bfloat16)
        if op == "w4a4_gemm":
            st["ga"], st["gw"] = float(x.abs().amax()) / (6 * 448), 0.75
            codes, s = _w4_codes(x, st["ga"])
            st["a"], st["a_scales"] = _pack4(codes), s.view(torch.uint8)
            # Weights as the packed format's own recipe draws them: every nibble, half-normal scales.
            st["w"] = torch.randint(0, 256, (N, K // 2), generator=gen, device=DEV, dtype=torch.uint8)
            st["w_scales"] = _e4m3(torch.randn((N, K // 16), generator=gen, device=DEV).abs() * 0.05).view(torch.uint8)
        else:
            q, st["a_scales"] = _a8_codes(x)
            st["a"] = q.view(torch.uint8)
            st["w"] = _e4m3(torch.randn((N, K), generator=gen, device=DEV) * 0.05).view(torch.uint8)
            st["w_scales"] = torch.rand(((N + 127) // 128, K // 128), generator=gen, device=DEV) * 1.5 + 0.5
        return st
    dtype = TYPES[case["type"]]
    st["x"] = _padded(M, K, pad, dtype)
    st["x"].copy_(_activations(M, K, gen))
    if op == "w4_quantize":
        st["g"] = float(st["x"].abs().amax()) / (6 * 448)
        st["g"] = float(torch.tensor(st["g"], dtype=torch.float32))
        st["out"] = (_bytes(M, K // 2), _bytes(M, K // 16))
        st["values"] = torch.empty((M, K), device=DEV)
    elif op == "a8_quantize" or case["out"] == "a8":
        st["out"] = (_bytes(M, K), torch.empty((M, K // 128), device=DEV))
    else:
        st["out"] = torch.empty((M, K), dtype=dtype, device=DEV)
    if op == "rms_norm":
        st["weight"] = (1.0 + 0.1 * torch.randn(K, generator=gen, device=DEV)).to(dtype)
        st["residual"] = st["residual_out"] = None
        if case["residual"]:
            st["residual"] = _padded(M, K, pad, dtype)
            st["residual"].copy_(4.0 * torch.randn((M, K), generator=gen, device=DEV))
            st["residual_out"] = torch.empty((M, K), dtype=dtype, device=DEV)
    return st


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    if op == "w4a4_gemm":
        return {"bytes": (M + case["N"]) * K * 9 / 16 + 2 * M * case["N"], "flops": 2 * M * case["N"] * K}
    if op == "w8a8_gemm":
        scales = 4 * (M + (case["N"] + 127) // 128) * (K // 128)
        return {"bytes": (M + case["N"]) * K + scales + 2 * M * case["N"], "flops": 2 * M * case["N"] * K}
    size = {"bf16": 2, "f16": 2, "f32": 4}[case["type"]]
    if op == "w4_quantize":                 # rows in; values in FP32 and scales out
        return {"bytes": M * K * (size + 4 + 1 / 16), "flops": 3 * M * K}
    if op == "a8_quantize":
        return {"bytes": M * K * (size + 1 + 1 / 32), "flops": 2 * M * K}
    written = 1 + 1 / 32 if case["out"] == "a8" else size
    return {"bytes": M * K * (size * (3 if case["residual"] else 1) + written) + K * size, "flops": 6 * M * K}


# ------------------------------------------------------------------ 64 bits
def _near_e4m3(v):
    """Nearest E4M3 value (ties to the even one), saturating, in 64 bits."""
    a = v.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))).clamp(-6, 8) - 3)
    return torch.sign(v) * torch.clamp(torch.round(a / step) * step, max=448.0)


def _near_e2m1(v):
    """Nearest E2M1 value (ties to the even one), saturating, in 64 bits."""
    a = v.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(v.dtype)
    return torch.sign(v) * torch.round(a / step) * step


def _exact_a8(y):
    M, K = y.shape
    amax = y.view(M, -1, 128).abs().amax(2).clamp_min(FLOOR)
    return _near_e4m3(y.view(M, -1, 128) * (448.0 / amax).unsqueeze(2)).view(M, K), amax / 448.0


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "w4a4_gemm":
        def deq(p, s):
            mags = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
            n = torch.empty((p.shape[0], 2 * p.shape[1]), dtype=torch.int32, device=DEV)
            n[:, 0::2], n[:, 1::2] = p & 15, p >> 4
            v = mags[n & 7] * (1 - 2 * (n >> 3))
            return (v.view(s.shape[0], -1, 16) * s.view(torch.float8_e4m3fn).double().unsqueeze(2)).view(v.shape)
        return deq(st["a"], st["a_scales"]) @ deq(st["w"], st["w_scales"]).t() * st["ga"] * st["gw"]
    if op == "w8a8_gemm":
        a = st["a"].view(torch.float8_e4m3fn).double() * st["a_scales"].double().repeat_interleave(128, 1)
        rows = torch.arange(case["N"], device=DEV) // 128
        w = st["w"].view(torch.float8_e4m3fn).double() * st["w_scales"].double()[rows].repeat_interleave(128, 1)
        return a @ w.t()
    x = st["x"].double()
    M, K = x.shape
    if op == "w4_quantize":
        xg = x.view(M, -1, 16) if x.is_contiguous() else x.contiguous().view(M, -1, 16)
        s = _near_e4m3(xg.abs().amax(2) / (6.0 * st["g"]))
        d = (s * st["g"]).float().double().unsqueeze(2)      # the group's scale is an FP32 number
        v = torch.where(d > 0, _near_e2m1(xg / torch.where(d > 0, d, 1.0)) * d, 0.0)
        return {"values": v.view(M, K), "scales": s}
    if op == "a8_quantize":
        q, s = _exact_a8(x.contiguous())
        return {"codes": q, "scales": s}
    got = {}
    if st["residual"] is not None:
        x = x + st["residual"].double()
        got["residual"] = x
    y = x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * st["weight"].double()
    if case["out"] == "a8":
        got["codes"], got["scales"] = _exact_a8(y.contiguous())
    else:
        got["y"] = y
    return got
