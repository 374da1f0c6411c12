"""The gradients of the layer of examples/layer_step.py against the same steps in 64
bits, with the same quantisations and roundings, and what that comparison notices."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import moe_ragged_contraction_gb300 as mx
import _layer_ref as L

# What may differ is where a rounding falls on the other side, as the sums before it are in fp32. A sum of 256 products is off
# by about sqrt(256) 2^-24 of its terms' size, 2^-12 of a bf16 step of 2^-8: with cancellation of a factor of ten, one value
# in a hundred falls to the neighbouring bf16 value, 2^-8 away, and one in 32 of those to the neighbouring E4M3
# value, 2^-3 away: sqrt(0.01) 2^-8 + sqrt(0.01 / 32) 2^-3 = 2.6e-3 in the norm a step. Four such steps follow one another at
# most: 1e-2. (The last rounding to bf16 is on both sides.)
LIMIT = 1e-2

T, E, H, I, K = 300, 4, 256, 128, 2


def inputs(seed):
    rng = np.random.default_rng(seed)
    f = lambda *shape: rng.standard_normal(shape).astype(np.float32)  # noqa: E731
    return L.rounded(f(T, H)).astype(np.float32), L.rounded(f(T, H)).astype(np.float32), f(E, H) / np.float32(16), f(E, 2 * I, H) / np.float32(16), f(E, H, I) / np.float32(11)


@pytest.mark.parametrize("change", [c for c in L.CHANGES if c != "second choice of a token"])
def test_a_term_left_out_is_far_outside_the_limit(change):
    args = inputs(1)
    want, got = L.layer(*args, K), L.layer(*args, K, change=change)
    assert max(L.distance(a, b) for a, b in zip(got, want)) > 3 * LIMIT


def test_a_single_pair_left_out_is_outside_the_limit():
    args = inputs(1)
    want, got = L.layer(*args, K), L.layer(*args, K, change="second choice of a token")
    assert L.distance(got[0][7], want[0][7]) > 3 * LIMIT and L.distance(got[1][7], want[1][7]) > 3 * LIMIT


@pytest.mark.gpu
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_against_the_same_steps_in_64_bits(seed):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "layer_step.py")
    spec = importlib.util.spec_from_file_location("layer_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    args = inputs(seed)
    want = L.layer(*args, K)
    x, dout, router, w13, w2 = (torch.from_numpy(a).cuda() for a in args)
    out, dx, (dw13, dw2, drouter) = m.layer(x.bfloat16(), dout.bfloat16(), router, w13, w2, K)
    for name, got, w in zip(("out", "dx", "dw13", "dw2", "drouter"), (out, dx, dw13, dw2, drouter), want):
        got = got.double().cpu().numpy()
        assert L.distance(got, w) <= LIMIT, name
        if name in ("out", "dx"):  # every token by itself: a few more of its roundings may fall otherwise
            rows = np.linalg.norm(got - w, axis=1) / np.linalg.norm(w, axis=1)
            assert rows.max() <= 3 * LIMIT, name
    assert mx.device_status(clear=True) == 0
