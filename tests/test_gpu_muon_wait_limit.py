"""The limit of the kernels' waits bounds a hand-over, not a call: an update that
runs three times as long as the limit, none of whose products or hand-overs does,
reports nothing. In a child process with a limit of 8 ms."""
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
gen.manual_seed(2)
# 1024 tiles of 256 x 256 in each product, 14 rounds of about 0.07 ms; 48 products
g = torch.randn(8192, 8192, generator=gen, device="cuda").bfloat16()
out = mx.muon_update(g, steps=16)
torch.cuda.synchronize()
assert mx.device_status(clear=True) == 0
t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
t0.record()
again = mx.muon_update(g, steps=16)
t1.record()
torch.cuda.synchronize()
ms = t0.elapsed_time(t1)
assert ms > 20, ms
assert mx.device_status(clear=True) == 0
assert torch.equal(out, again) and torch.isfinite(out).all()
print("OK", ms)
'''


def test_calls_longer_than_the_limit():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    env = dict(os.environ, MXFP8_WAIT_LIMIT_MS="8")
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "OK" in r.stdout, r.stdout + r.stderr
