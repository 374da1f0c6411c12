"""The limit of wgrad_main's waits bounds a hand-over, not a call: a call that
runs half as long again as the limit, none of whose tiles does, reports nothing. In a
child process with a limit of 3 ms."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import sys
import torch
sys.path.insert(0, sys.argv[1])
import moe_ragged_contraction_gb300 as mx
gen = torch.Generator(device="cuda")
gen.manual_seed(1)
E, N, K, M = 32, 7168, 2048, 524288  # tiles of about 0.09 ms
def operand(rows):
    q = torch.randint(0, 0x58, (rows, M), dtype=torch.uint8, device="cuda", generator=gen)
    q |= torch.randint(0, 2, (rows, M), dtype=torch.uint8, device="cuda", generator=gen) << 7
    return q, torch.randint(124, 131, (rows, M // 32), dtype=torch.uint8, device="cuda", generator=gen)
A, sA = operand(N)
B, sB = operand(K)
offs = (torch.arange(1, E + 1, device="cuda") * (M // E)).int()
out = mx.wgrad_grouped(A, sA, B, sB, offs)
torch.cuda.synchronize()
assert mx.device_status(clear=True) == 0, "status"
t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
t0.record()
again = mx.wgrad_grouped(A, sA, B, sB, offs)
t1.record()
torch.cuda.synchronize()
ms = t0.elapsed_time(t1)
assert ms > 4, ms
assert mx.device_status(clear=True) == 0, "status"
assert torch.equal(out, again) and torch.isfinite(out).all()
print("OK", ms)
'''


def test_calls_longer_than_the_limit():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    env = dict(os.environ, MXFP8_WAIT_LIMIT_MS="3")
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "OK" in r.stdout, r.stdout + r.stderr
