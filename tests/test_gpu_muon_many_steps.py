"""The error of muon_update with the default coefficients over many steps.

Tolerance (derived). One step's roundings to 11 bits come to about 0.9e-3 of the
norm as independent errors. A later step multiplies an error along a singular
value s by the derivative a + 3 b s^2 + 5 c s^4. Its mean logarithm over the
values that occur is about 0.2 in the first steps, where the signal grows too, and
negative from the sixth on (-0.1 .. -0.4): the errors do not grow on average. If
those of all steps line up they come to steps x 0.9e-3, and bf16 adds 1.1e-3.
That holds for matrices of full rank: directions without a part in u are noise
after some ten steps of 3.4 each, in fp32 as well."""
import numpy as np
import pytest
import torch

import moe_ragged_contraction_gb300 as mx
from _experts_ref import muon

pytestmark = pytest.mark.gpu


def spectrum(m, n, kind, rng):
    g = rng.standard_normal((m, n))
    if kind == "strong":
        g = g + 3 * rng.standard_normal((m, 4)) @ rng.standard_normal((4, n))
    elif kind == "decay":
        u, _ = np.linalg.qr(rng.standard_normal((m, m)))
        v, _ = np.linalg.qr(rng.standard_normal((n, m)))
        g = (u * np.logspace(0, -3, m)) @ v.T
    return (g * 1e-3).astype(np.float32)


@pytest.mark.parametrize("steps", [8, 12, 16])
@pytest.mark.parametrize("kind", ["normal", "strong", "decay"])
@pytest.mark.parametrize("shape", [(100, 264), (200, 328), (384, 160), (331, 1000)])  # on chip, general, tall, odd
def test_default_coefficients(shape, kind, steps):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.build()
    m, n = sorted(shape)
    g = spectrum(m, n, kind, np.random.default_rng(m + steps))
    g = np.ascontiguousarray(g if shape[0] < shape[1] else g.T)[None]
    out = mx.muon_update(torch.from_numpy(g).cuda(), steps=steps).float().cpu().numpy()
    want = muon(g, steps=steps)[0]
    assert np.linalg.norm(out - want) <= (steps * 0.9e-3 + 1.1e-3) * np.linalg.norm(want)
    assert mx.device_status(clear=True) == 0
