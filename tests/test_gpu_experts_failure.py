"""Failure detection of the expert-weight operators without a GPU fault: a
host-side test hook makes the first pipeline stage declare more bytes than it
receives, so that its bounded wait runs out. The kernel must stop, raise
MXFP8_DEV_WAIT_TIMEOUT and return (whatever waits on its work runs out too); the
context stays usable and the next call is correct. Runs in a child process with
a 50 ms wait limit."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import ctypes, sys
import torch
sys.path.insert(0, sys.argv[1])
import moe_ragged_contraction_gb300 as mx
lib = mx.load()
lib.mxfp8_test_stall_next_call.argtypes = [ctypes.c_int]
gen = torch.Generator(device="cuda")
gen.manual_seed(1)
rand = lambda *s: torch.randn(s, generator=gen, device="cuda")
E, H, I = 6, 512, 256
w13, s13 = mx.quantize_tokenwise(rand(E * 2 * I, H))
w2, s2 = mx.quantize_tokenwise(rand(E * H, I))
args = (rand(12, H).bfloat16(), rand(E, H).bfloat16(), w13.view(E, 2 * I, H), s13.view(E, 2 * I, -1), w2.view(E, H, I), s2.view(E, H, -1), 3)
g = rand(3, 300, 520)
for call in (lambda: mx.moe_layer(*args), lambda: mx.muon_update(g)):
    mx.device_status(clear=True)
    want = call()
    torch.cuda.synchronize()
    assert mx.device_status(clear=True) == 0
    lib.mxfp8_test_stall_next_call(1)
    call()
    torch.cuda.synchronize()
    st = mx.device_status(clear=True)
    assert st & 8, f"expected the wait-timeout bit, status={st}"
    got = call()
    torch.cuda.synchronize()
    assert mx.device_status(clear=True) == 0 and torch.equal(got, want)
print("OK")
'''


def test_wait_timeout_reported_and_context_survives():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    env = dict(os.environ, MXFP8_WAIT_LIMIT_MS="50")
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "OK" in r.stdout, r.stdout + r.stderr
