"""Matrices whose squares leave fp32's range below: the norm of muon_update holds
as long as the elements do. Powers of two change nothing at eps = 0, down to
elements whose squares are zero in fp32; and against 64 bits with an eps of the
same order."""
import numpy as np
import pytest
import torch

import moe_ragged_contraction_gb300 as mx
from _experts_ref import muon

pytestmark = pytest.mark.gpu

# one cluster a matrix (one CTA, two); the general path, wide, tall, in pieces
SHAPES = [(2, 96, 136), (1, 40, 520), (2, 264, 328), (1, 328, 152), (1, 130, 2600)]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.build()
    mx.device_status(clear=True)


def gradient(E, N, K):
    """Elements of 2^-10 .. 1 in magnitude, so that scaling by 2^-115 keeps them normal."""
    rng = np.random.default_rng(N + K)
    g = rng.standard_normal((E, N, K))
    return (np.sign(g) * np.clip(np.abs(g), 2.0 ** -10, 1.0)).astype(np.float32)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("momentum", [False, True])
def test_powers_of_two_change_nothing(shape, momentum):
    g = torch.from_numpy(gradient(*shape)).cuda()
    m = torch.from_numpy(gradient(*shape)).cuda().flip(1).contiguous() if momentum else None
    run = lambda s: mx.muon_update(g * s, None if m is None else m * s, mu=0.5, eps=0.0)  # noqa: E731 (mu a power of two: exact sums scale exactly)
    want = run(1.0)
    assert torch.isfinite(want).all()
    for p in (20, -20, -40, -45, -50, -60, -80, -100, *(() if momentum else (-115,))):  # (below, the momentum's sums lose bits)
        assert torch.equal(run(2.0 ** p), want), p
    assert mx.device_status(clear=True) == 0


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("p,eps", [(-70, 1e-20), (-70, 1e-35), (-110, 1e-32), (-30, 0.0)])
def test_small_values_against_64_bits(shape, p, eps):
    """The tolerance of the iteration at usual scales (a step's roundings twice over, and bf16's): 4.5e-3."""
    g = gradient(*shape) * np.float32(2.0 ** p)
    out = mx.muon_update(torch.from_numpy(g).cuda(), eps=eps).float().cpu().numpy()
    want = muon(g, eps=float(np.float32(eps)))[0]
    for e in range(len(g)):
        assert np.linalg.norm(out[e] - want[e]) <= 4.5e-3 * np.linalg.norm(want[e])


def test_smallest_values():
    """Subnormal elements, a single non-zero element, zeros beside them."""
    for shape in ((3, 48, 64), (3, 144, 160)):
        g = np.zeros(shape, np.float32)
        g[0, 5, 7] = 2.0 ** -149
        g[1, 3, 1], g[1, 4, 2] = 2.0 ** -140, -(2.0 ** -140)
        out = mx.muon_update(torch.from_numpy(g).cuda(), eps=0.0).float().cpu().numpy()
        p1 = lambda s: 3.4445 * s - 4.7750 * s ** 3 + 2.0315 * s ** 5  # noqa: E731
        for e, start in ((0, 1.0), (1, 0.5 ** 0.5)):
            s = start
            for _ in range(5):
                s = p1(s)
            at = np.nonzero(g[e])
            assert np.allclose(np.abs(out[e][at]), abs(s), rtol=4.5e-3) and np.count_nonzero(out[e]) == len(at[0])
        assert not out[2].any()
        # beside the default eps: about a^5 u / eps, below 2^-107 here; the general path's planes end at 2^-35
        tiny = mx.muon_update(torch.from_numpy(g).cuda())
        assert float(tiny.abs().max()) <= 2.0 ** -107 and not tiny[2].any()
