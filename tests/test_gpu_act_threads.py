"""The quantised-activation entries called for the first time in a process by several host threads at once, each with
its own stream, inputs and outputs: they race to fill the kernels' attributes, the table of resident clusters and the
tensor maps. Every result equals the same call made alone afterwards, bit for bit."""
from __future__ import annotations

import os
import subprocess
import sys
import threading

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
THREADS, REPEATS = 6, 4
# (M, N, K): few rows with K split, many tiles, many rows of each tile width and orientation.
SHAPES = [(1, 640, 2560), (40, 256, 5120), (33, 20000, 256), (200, 1280, 2560), (300, 5000, 512), (128, 20224, 512)]


def calls(seed):
    """Every entry on every shape, on the current stream's thread's own tensors: functions that return tensors."""
    import torch

    import weight_only_quantized_packed_gb300 as wqp

    g = torch.Generator(device="cuda").manual_seed(seed)
    made = []
    for M, N, K in SHAPES:
        x, r = (torch.randn((M, K), generator=g, device="cuda").bfloat16() for _ in range(2))
        ones = torch.ones(K, device="cuda").bfloat16()
        code = lambda *s: torch.randint(0, 119, s, generator=g, device="cuda", dtype=torch.uint8)
        a4, sa4, w4, sw4 = code(M, K // 2), code(M, K // 16), code(N, K // 2), code(N, K // 16)
        a8, w8 = code(M, K), code(N, K)
        sa8, sw8 = (torch.rand((n, K // 128), generator=g, device="cuda") for n in (M, (N + 127) // 128))
        made += [lambda x=x: wqp.w4_quantize(x, 0.01), lambda x=x: wqp.a8_quantize(x),
                 lambda x=x, r=r, w=ones: wqp.rms_norm(x, w, 1e-6, residual=r), lambda x=x, r=r, w=ones: wqp.rms_norm_a8(x, w, 1e-6, residual=r),
                 lambda a=(a4, sa4, w4, sw4, N, K): (wqp.w4a4_gemm(*a),), lambda a=(a8, sa8, w8, sw8, N, K): (wqp.w8a8_gemm(*a),)]
    return made


def race():
    import torch

    import weight_only_quantized_packed_gb300 as wqp

    work = [calls(100 + i) for i in range(THREADS)]
    torch.cuda.synchronize()
    results, errors, start = [None] * THREADS, [], threading.Barrier(THREADS)

    def worker(i):
        try:
            stream = torch.cuda.Stream()
            start.wait()
            with torch.cuda.stream(stream):
                for n in range(REPEATS):
                    order = work[i] if n else work[i][i:] + work[i][:i]        # not all at the same entry
                    got = [[t.clone() for t in f()] for f in order]
                    results[i] = got if n else None
            stream.synchronize()
        except Exception as e:   # noqa: BLE001 - reported below with its thread
            errors.append((i, repr(e)))

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(THREADS)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=300)
    assert not any(t.is_alive() for t in threads), "a thread did not finish"
    assert not errors, errors[:4]
    for i in range(THREADS):
        for j, f in enumerate(work[i]):
            alone = f()
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(alone, results[i][j])), (i, j)
    assert wqp.get_device_error() == 0


def test_threads_race_on_first_calls():
    """In a process of its own, in which no entry was called before."""
    done = subprocess.run([sys.executable, "-c", "from tests.test_gpu_act_threads import race; race(); print('raced')"], cwd=ROOT,
                          capture_output=True, text=True, timeout=600)
    assert done.returncode == 0 and "raced" in done.stdout, done.stdout[-2000:] + done.stderr[-4000:]
