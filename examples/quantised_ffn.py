"""A feed-forward block whose activations are quantised too, next to the same block with BF16 activations.

    python examples/quantised_ffn.py [--hidden 5120 --ffn 17408 --rows 1,64,2048]

The weights are made here with the library's own quantisers: gate and up as W8A16 matrices, down as a W4A16 matrix.
For each number of rows the block runs as a serving program would run it,

    codes, scales, h = rms_norm_a8(x, weight, eps, residual)        norm, residual's addition, 8-bit rows
    u = w8a8_gemm(codes, scales, gate_up)                           8-bit product
    q, qs = w4_quantize(silu(gate) * up, g)                         4-bit rows
    y = w4a4_gemm(q, qs, down)                                      4-bit product

and as it runs without quantised activations (rms_norm, w8a16_gemm, w4a16_gemm_tc), and prints how far apart the two
outputs are and what each takes.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_only_quantized_packed_gb300 as wqp  # noqa: E402

EPS = 1e-6


class FeedForward:
    """Random-init packed weights of one block."""

    def __init__(self, hidden: int, ffn: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.ffn = hidden, ffn
        self.norm = (1 + 0.1 * torch.randn(hidden, generator=g, device="cuda")).bfloat16()
        # W8A16: E4M3 with a scale per 128x128 block; each block's largest magnitude becomes 448.
        w = torch.randn((2 * ffn, hidden), generator=g, device="cuda") * hidden ** -0.5
        blocks = w.view(2 * ffn // 128, 128, hidden // 128, 128)
        self.gate_up_scales = (blocks.abs().amax((1, 3)) / 448).contiguous()
        q = blocks / self.gate_up_scales[:, None, :, None]
        self.gate_up = q.view(2 * ffn, hidden).to(torch.float8_e4m3fn).view(torch.uint8)
        # W4A16: the library's quantiser, under one global scale.
        w = torch.randn((hidden, ffn), generator=g, device="cuda") * ffn ** -0.5
        self.down_global = float(w.abs().amax()) / (6 * 448)
        self.down, self.down_scales = wqp.w4_quantize(w, self.down_global)

    def act(self, u):
        gate, up = u[:, :self.ffn], u[:, self.ffn:]
        return torch.nn.functional.silu(gate) * up

    def quantised(self, x, residual, act_global: float):
        codes, scales, h = wqp.rms_norm_a8(x, self.norm, EPS, residual=residual)
        u = wqp.w8a8_gemm(codes, scales, self.gate_up, self.gate_up_scales, 2 * self.ffn, self.hidden)
        q, qs = wqp.w4_quantize(self.act(u), act_global)
        return wqp.w4a4_gemm(q, qs, self.down, self.down_scales, self.hidden, self.ffn, act_global, self.down_global), h

    def bf16_activations(self, x, residual):
        y, h = wqp.rms_norm(x, self.norm, EPS, residual=residual)
        u = wqp.w8a16_gemm(y, self.gate_up, self.gate_up_scales, 2 * self.ffn, self.hidden)
        a = self.act(u)
        return wqp.w4a16_gemm_tc(a, self.down, self.down_scales, self.hidden, self.ffn, self.down_global), h, float(a.abs().amax())


def timed(call, reps: int = 10) -> float:
    """Microseconds a call, warm."""
    for _ in range(3):
        call()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(reps):
        call()
    end.record()
    end.synchronize()
    return start.elapsed_time(end) / reps * 1e3


def main(argv=None) -> list:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--hidden", type=int, default=5120)
    ap.add_argument("--ffn", type=int, default=17408)
    ap.add_argument("--rows", default="1,64,2048")
    a = ap.parse_args(argv)
    block, found = FeedForward(a.hidden, a.ffn), []
    for rows in (int(r) for r in a.rows.split(",")):
        g = torch.Generator(device="cuda").manual_seed(rows)
        x = torch.randn((rows, a.hidden), generator=g, device="cuda").bfloat16()
        residual = torch.randn((rows, a.hidden), generator=g, device="cuda").bfloat16()
        want, h, amax = block.bf16_activations(x, residual)
        g4 = amax / (6 * 448)                        # calibrated once, as a serving program would
        got, h8 = block.quantised(x, residual, g4)
        off = float((got.float() - want.float()).norm() / want.float().norm())
        assert torch.equal(h, h8)
        t8, t16 = timed(lambda: block.quantised(x, residual, g4)), timed(lambda: block.bf16_activations(x, residual))
        print(f"{rows:5d} rows: quantised activations {t8:9.1f} us, BF16 activations {t16:9.1f} us, outputs {off:.3f} apart")
        found.append((rows, off, t8, t16))
    return found


if __name__ == "__main__":
    main()
