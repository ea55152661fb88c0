"""Calls from host threads that have made no CUDA call before, and that use a kernel first with different amounts of shared
memory at the same time; in a process of their own."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import threading
import torch
import hadamard_rotation_gb300 as hq

def grouped(E):
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    args = (u8(8, 32), u8(8, 2), u8(E, 40, 32), u8(E, 512), off)
    return lambda: hq.hq_grouped_gemm_mxfp4(*args)

def lora(M, R):
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    args = (u8(M, 32), u8(M, 2), u8(40, 32), u8(512), bf(M, 64), bf(3, R, 64), bf(3, 40, R), torch.ones(3, device="cuda"),
            torch.zeros(M, dtype=torch.int32, device="cuda"))
    return lambda: hq.hq_lora_gemm_mxfp4(*args)

def wgrad():
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    args = (u8(40, 64), u8(512), u8(32, 64), u8(512), torch.tensor([0, 128], dtype=torch.int32, device="cuda"))
    return lambda: hq.hq_grouped_wgrad_mxfp4(*args)

def norm(M, D):
    h, y = torch.ones(M, D, device="cuda"), torch.ones(M, D, device="cuda")
    return lambda: hq.hq_block_norm(h, y)

def int8(K):
    x = torch.ones(64, K, device="cuda")
    return lambda: hq.hq_rotate_quant_int8(x, 16)

calls = [grouped(1), grouped(512), wgrad(), lora(1, 8), lora(128, 128), norm(3, 64), norm(3, 4096), norm(500, 2048), int8(40960), int8(110592)]
torch.cuda.synchronize()
bad, gate = [], threading.Barrier(len(calls))

def work(f):
    gate.wait()
    for _ in range(200):
        try:
            f()
        except Exception as e:
            bad.append(repr(e))

threads = [threading.Thread(target=work, args=(f,)) for f in calls]
for t in threads: t.start()
for t in threads: t.join()
torch.cuda.synchronize()
assert not bad, (len(bad), bad[:3])
assert hq.hq_read_fault() == 0
print("ok")
"""


def test_first_calls_of_several_threads():
    from hadamard_rotation_gb300 import build

    build.build()
    out = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip().endswith("ok"), (out.stdout[-1000:], out.stderr[-3000:])
