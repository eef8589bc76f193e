"""The experts' entries called for the first time in a process by several host threads at once, each with its own
stream, inputs and outputs: they race to fill the kernels' attributes and the tensor maps. Every result equals the same
call made alone afterwards, bit for bit."""
from __future__ import annotations

import os
import subprocess
import sys
import threading

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
THREADS, REPEATS = 6, 4


def race():
    import torch

    import weight_only_quantized_packed_gb300 as wqp
    from tests.test_gpu_experts import Block

    blocks, inputs = [Block(512, 256, 16, 4, seed=10 * i) for i in range(THREADS)], []
    for i in range(THREADS):
        g = torch.Generator(device="cuda").manual_seed(i)
        inputs.append([[torch.randn((T, 512), generator=g, device="cuda").bfloat16() for _ in range(2)] for T in (1, 5, 300)])
    torch.cuda.synchronize()
    results, errors, start = [None] * THREADS, [], threading.Barrier(THREADS)

    def worker(i):
        try:
            stream = torch.cuda.Stream()
            start.wait()
            with torch.cuda.stream(stream):
                for _ in range(REPEATS):
                    results[i] = [[t.clone() for t in blocks[i](*x)] for x in inputs[i]]
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
        for x, got in zip(inputs[i], results[i]):
            assert all(torch.equal(a, b) for a, b in zip(blocks[i](*x), got)), i
    assert wqp.get_device_error() == 0


def test_threads_race_on_first_calls():
    """In a process of its own, in which no entry was called before."""
    done = subprocess.run([sys.executable, "-c", "from tests.test_gpu_experts_threads import race; race(); print('raced')"], cwd=ROOT,
                          capture_output=True, text=True, timeout=600)
    assert done.returncode == 0 and "raced" in done.stdout, done.stdout[-2000:] + done.stderr[-4000:]
