"""Updates of small matrices stay on chip and take no scratch: the query asks for
a nominal amount, the cache holds none, a call can be captured on a stream that
has run nothing before."""
import os
import subprocess
import sys

import pytest

import moe_ragged_contraction_gb300 as mx

NOMINAL = 512


@pytest.mark.parametrize("E,N,K", [(1, 1, 8), (4, 128, 256), (2, 2048, 128), (2048, 128, 2048)])
def test_small_matrices_ask_for_a_nominal_amount(E, N, K):
    mx.build()
    assert mx.muon_update_workspace_bytes(E, N, K) == NOMINAL
    assert mx.muon_update_workspace_bytes(E, 136, 136) > NOMINAL


CHILD = r"""
import sys
import torch
sys.path.insert(0, sys.argv[1])
import moe_ragged_contraction_gb300 as mx
gen = torch.Generator(device="cuda")
gen.manual_seed(4)
g = torch.randn(5, 72, 264, generator=gen, device="cuda")
want = mx.muon_update(g)  # (loads the kernel)
ws = torch.empty(int(sys.argv[2]), dtype=torch.uint8, device="cuda")
assert torch.equal(mx.muon_update(g, workspace=ws), want)
torch.cuda.synchronize()
out, other = torch.zeros_like(want), torch.zeros(1, 136, 136, device="cuda")
other_out = torch.empty(1, 136, 136, dtype=torch.bfloat16, device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):  # on a stream that has run nothing
    mx.muon_update(g, out=out)
    try:
        mx.muon_update(other, out=other_out)
        raise SystemExit("a larger matrix needs scratch that the stream does not have")
    except mx.Mxfp8Error as e:
        assert e.code == -5
graph.replay()
torch.cuda.synchronize()
assert torch.equal(out, want) and mx.device_status(clear=True) == 0
print("OK")
"""


@pytest.mark.gpu
def test_capture_on_a_fresh_stream():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.build()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CHILD, root, str(NOMINAL)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "OK" in r.stdout, r.stdout + r.stderr
