"""Coefficients of muon_update that would take the iteration out of the range
of its fp16 operands are refused on the host; those inside are computed.

A step takes a singular value s to a s + b s^3 + c s^5, and any s in [0, 1] can
occur in the first one. A = X X^T has the eigenvalues s^2 and R = b A + c A A -
beta I the values b s^2 + c s^4 - beta (beta: 0.875 (b + c) in the last step, half of
that in the one before); both are stored as fp16 times 4096, which ends at 16."""
import numpy as np
import pytest

import moe_ragged_contraction_gb300 as mx
from moe_ragged_contraction_gb300 import _lib
from _experts_ref import muon as muon64

P = 0x10000  # 256-byte aligned fake address: never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    mx.build()
    return mx.load()


def largest(a, b, c, steps, grid=20001):
    """The largest magnitude in A or R over the whole iteration, from a grid of singular values."""
    worst, top = 0.0, 1.0
    for k in range(steps):
        s = np.linspace(0.0, top, grid)
        beta = (b + c) * (0.875 if k + 1 == steps else 0.4375 if k + 2 == steps else 0.0)
        worst = max(worst, top * top, np.abs(b * s ** 2 + c * s ** 4 - beta).max())
        if k + 1 < steps:
            top = np.abs(a * s + b * s ** 3 + c * s ** 5).max()
            if not top < 1e6:
                return np.inf
    return worst


def verdict(lib, coeffs, steps):
    # E = 0 is a no-op once the arguments are accepted: no GPU is needed
    return lib.mxfp8_muon_update(P, 0, None, 0, 16, 24, 0.9, 1, steps, *coeffs, 1e-7, P, None)


@pytest.mark.parametrize("coeffs,steps", [
    ((4.0, 0.0, 0.0), 3), ((3.0, 0.0, 0.0), 3), ((4.5, -0.2, 0.0), 2), ((2.5, -0.1, 0.0), 3), ((1.0, 0.0, 16.0), 2),
    ((16.0, 16.0, 16.0), 16), ((-4.0, 0.0, 0.0), 2), ((0.0, 8.0, 12.0), 1),
])
def test_out_of_range_is_refused(lib, coeffs, steps):
    assert largest(*coeffs, steps) >= 16
    assert verdict(lib, coeffs, steps) == _lib.EINVAL
    assert b"range" in lib.mxfp8_last_error()


@pytest.mark.parametrize("coeffs", [(3.4445, -4.7750, 2.0315), (1.5, -0.5, 0.0), (15 / 8, -10 / 8, 3 / 8), (2.0, -1.5, 0.5), (3.0, -3.2, 1.2)])
def test_usual_coefficients_are_taken_for_every_step_count(lib, coeffs):
    for steps in range(1, 17):
        assert verdict(lib, coeffs, steps) == _lib.OK


def test_verdict_follows_the_largest_value(lib):
    """Refused wherever the exact iteration leaves the range, taken wherever it stays well inside."""
    rng = np.random.default_rng(0)
    seen = {"in": 0, "out": 0}
    for _ in range(400):
        coeffs, steps = tuple(float(np.float32(v)) for v in rng.uniform(-6, 6, 3)), int(rng.integers(1, 6))
        worst = largest(*coeffs, steps, grid=2001)
        if worst >= 16:
            assert verdict(lib, coeffs, steps) == _lib.EINVAL, (coeffs, steps, worst)
            seen["out"] += 1
        elif worst < 8:
            assert verdict(lib, coeffs, steps) == _lib.OK, (coeffs, steps, worst)
            seen["in"] += 1
    assert min(seen.values()) > 40


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1, 72, 104), (1, 152, 264), (1, 264, 136)])
@pytest.mark.parametrize("coeffs,steps", [((3.7, 0.0, 0.0), 2), ((1.0, 13.0, 0.0), 1), ((3.3, 0.2, 0.0), 2)])
def test_just_inside_the_range(lib, coeffs, steps, shape):
    """A matrix of rank one has the singular value 1 after the division by its norm: A or R come to 10 .. 14 there.
    Its roundings to 11 bits (R, X in R X, A) come to at most 3 * 2^-11 of the largest term, here at most four times the result,
    and bf16 adds 2^-9: 8e-3 of the norm."""
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    assert 10 < largest(*coeffs, steps) < 14
    rng = np.random.default_rng(shape[1])
    g = (rng.standard_normal((shape[0], shape[1], 1)) * rng.standard_normal((shape[0], 1, shape[2])) * 1e-2).astype(np.float32)
    out = mx.muon_update(torch.from_numpy(g).cuda(), steps=steps, coeffs=coeffs).float().cpu().numpy()
    want = muon64(g, steps=steps, coeffs=coeffs)[0]
    assert np.linalg.norm(out - want) <= 8e-3 * np.linalg.norm(want)
    assert mx.device_status(clear=True) == 0
