"""The orthogonalised update (muon_update) against a 64-bit implementation on
the host: wide, tall, square and tiny matrices, every type, momentum forms,
step counts and coefficients, spectra from flat to rank one, zero and non-finite
matrices, streams, CUDA graphs, and the refusals.

Tolerance (derived). Each step rounds X, A and R to 11 significant bits, an
error of at most 2^-12 of each element, 2^-12 / sqrt(3) of its norm on average.
A step X <- a X + (b A + c A A) X whose largest singular value is near 1
multiplies an error in X by up to |a| + 3 |b| + 5 |c| = 28 for one that meets
every term alone, but the terms cancel: the derivative of a s + b s^3 + c s^5 is
at most 3.45 in magnitude on the s in [0, 1.2] that occur, and below 2.4 for
s > 0.6, where the last steps work. With 2.8 as the largest eigenvalue of R, the
roundings made in one step come to at most 2^-12 / sqrt(3) * (2.8 (R) + 2.8 (X
in R X) + 4.8 * 1.2 (A)) = 1.6e-3 if they all line up, about 0.9e-3 as
independent errors; errors of earlier steps pass later ones with the factors
above while the signal grows alike. Twice 1.6e-3, with bf16's rounding of the
result (2^-9 / sqrt(3) = 1.1e-3) on top: 4.5e-3 in the 2-norm, and no element
further off than a tenth of the root mean square plus that bound of its size.
"""
import numpy as np
import pytest
import torch

import moe_ragged_contraction_gb300 as mx
from _experts_ref import bf16_round, muon

pytestmark = pytest.mark.gpu
REL = 4.5e-3


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.build()
    mx.load()
    mx.device_status(clear=True)


def cuda(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t.to(dtype) if dtype else t


def gradient(E, N, K, seed, kind="normal"):
    rng = np.random.default_rng(seed)
    g = rng.standard_normal((E, N, K))
    if kind == "heavy":
        g = rng.standard_t(3, (E, N, K))
    elif kind == "decay":
        m = min(N, K)
        u, _ = np.linalg.qr(rng.standard_normal((E, N, m)))
        v, _ = np.linalg.qr(rng.standard_normal((E, K, m)))
        g = np.einsum("enm,m,ekm->enk", u, np.logspace(0, -3, m), v)
    elif kind == "lowrank":
        g = rng.standard_normal((E, N, 3)) @ rng.standard_normal((E, 3, K))
    elif kind == "strong":
        g = g + 3 * rng.standard_normal((E, N, 4)) @ rng.standard_normal((E, 4, K))
    return (g * 1e-3).astype(np.float32)


def close(got, want):
    g = got.float().cpu().numpy().astype(np.float64)
    for e in range(len(want)):
        n = np.linalg.norm(want[e])
        if n == 0:
            assert not g[e].any()
            continue
        assert np.linalg.norm(g[e] - want[e]) <= REL * n, np.linalg.norm(g[e] - want[e]) / n
        rms = n / np.sqrt(want[e].size)
        assert np.max(np.abs(g[e] - want[e]) - REL * np.abs(want[e])) <= 0.1 * rms


@pytest.mark.parametrize("E,N,K", [
    (1, 1, 8), (1, 8, 8), (2, 3, 16), (1, 1, 1000), (1, 999, 8),   # far smaller than a tile
    (4, 128, 256), (3, 331, 1000), (2, 1000, 328), (2, 256, 256), (1, 257, 264), (1, 255, 248), (5, 511, 520),
    (1, 65, 2048), (2, 2049, 64),
])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_against_64_bits(E, N, K, dtype):
    g = gradient(E, N, K, seed=E + N + K)
    if dtype == "bf16":
        g = bf16_round(g)
    m0 = gradient(E, N, K, seed=99) * 4
    gd, md = cuda(g, torch.bfloat16 if dtype == "bf16" else None), cuda(m0)
    out = mx.muon_update(gd, md)
    torch.cuda.synchronize()
    want, m1 = muon(g, m0)
    close(out, want)
    assert np.allclose(md.cpu().numpy(), m1, rtol=2e-6, atol=1e-9)
    again = mx.muon_update(gd, cuda(m0))
    assert torch.equal(out, again)
    assert mx.device_status(clear=True) == 0


@pytest.mark.parametrize("kind", ["heavy", "decay", "lowrank", "strong"])
@pytest.mark.parametrize("N,K", [(200, 328), (384, 160), (256, 256)])
def test_spectra(kind, N, K):
    g = gradient(2, N, K, seed=3, kind=kind)
    out = mx.muon_update(cuda(g))
    close(out, muon(g)[0])


@pytest.mark.parametrize("kw", [
    dict(steps=1), dict(steps=2), dict(steps=3), dict(steps=8), dict(coeffs=(1.5, -0.5, 0.0), steps=12),
    dict(coeffs=(15 / 8, -10 / 8, 3 / 8), steps=6), dict(nesterov=False), dict(mu=0.0), dict(eps=1.0),
])
def test_options(kw):
    g, m0 = gradient(2, 168, 296, seed=4, kind="strong"), gradient(2, 168, 296, seed=5)
    md = cuda(m0)
    out = mx.muon_update(cuda(g), md, **kw)
    want, m1 = muon(g, m0, **kw)
    close(out, want)
    assert np.allclose(md.cpu().numpy(), m1, rtol=2e-6, atol=1e-9)


def test_result_is_orthogonal():
    """A converging iteration: the rows become orthonormal, whatever the input (no reference needed)."""
    g = gradient(3, 120, 400, seed=6, kind="strong")
    out = mx.muon_update(cuda(g), coeffs=(1.5, -0.5, 0.0), steps=16).float()
    gram = out @ out.mT
    assert float((gram - torch.eye(120, device="cuda")).abs().max()) < 0.01


def test_scale_invariance_is_exact_for_powers_of_two():
    g = gradient(1, 96, 136, seed=7)
    a = mx.muon_update(cuda(g), eps=0.0)
    b = mx.muon_update(cuda(g * 2.0 ** 20), eps=0.0)
    assert torch.equal(a, b)


def test_zero_and_non_finite_matrices_stay_apart():
    g = bf16_round(gradient(6, 72, 104, seed=8))
    clean = mx.muon_update(cuda(g, torch.bfloat16))
    g[1] = 0
    g[3, 5, 7] = np.nan
    g[4, 0, 0] = np.inf
    out = mx.muon_update(cuda(g, torch.bfloat16))
    keep = [0, 2, 5]
    assert torch.equal(out[keep], clean[keep])
    assert not out[1].any()
    assert torch.isnan(out[3]).all() and torch.isnan(out[4]).all()
    assert not mx.muon_update(torch.zeros(2, 40, 64, device="cuda"), eps=0.0).any()
    big = torch.full((1, 16, 16), 3e30, device="cuda")
    assert torch.isnan(mx.muon_update(big)).all()  # the sum of squares overflows: NaN, not a wrong direction
    assert mx.device_status(clear=True) == 0


def test_one_matrix_and_out():
    g = gradient(1, 64, 200, seed=9)
    a = mx.muon_update(cuda(g))
    out = torch.empty(64, 200, dtype=torch.bfloat16, device="cuda")
    b = mx.muon_update(cuda(g[0]), out=out)
    assert b is out and torch.equal(a[0], b)


@pytest.mark.parametrize("E,N,K", [
    (1, 130, 2600), (2, 260, 2104), (1, 2111, 136),   # few long tiles: the contraction of X X^T in pieces
    (3, 100, 2056), (1, 4097, 96),                    # too long for one cluster by a little, and tall
    (2, 128, 2048), (1, 2048, 8), (7, 77, 520),       # one cluster a matrix: its largest size, its thinnest, three CTAs
    (90, 40, 264),                                    # more clusters than fit at once
])
def test_long_matrices(E, N, K):
    g = bf16_round(gradient(E, N, K, seed=N + K, kind="strong"))
    out = mx.muon_update(cuda(g, torch.bfloat16))
    close(out, muon(g)[0])
    assert torch.equal(out, mx.muon_update(cuda(g, torch.bfloat16)))
    assert mx.device_status(clear=True) == 0


@pytest.mark.parametrize("E,N,K", [
    (22, 264, 520), (23, 264, 520), (23, 520, 264),   # 132 tiles of 256 x 256: halved; 138: whole, wide and tall
    (12, 777, 1032), (9, 1100, 600), (35, 257, 257 + 7),
])
def test_many_tiles(E, N, K):
    g = bf16_round(gradient(E, N, K, seed=E + N, kind="strong"))
    m0 = gradient(E, N, K, seed=E)
    g[E // 2] = 0
    m0[E // 2] = 0
    gd, md = cuda(g, torch.bfloat16), cuda(m0)
    out = mx.muon_update(gd, md)
    want, m1 = muon(g, m0)
    close(out, want)
    assert np.allclose(md.cpu().numpy(), m1, rtol=2e-6, atol=1e-9)
    assert torch.equal(out, mx.muon_update(gd, cuda(m0)))
    assert mx.device_status(clear=True) == 0


@pytest.mark.parametrize("N,K", [(40, 96), (96, 40), (300, 200), (200, 304)])
def test_one_step_against_differences(N, K):
    """One step is odd in u and its derivative at u in direction d is what the formula's differences give."""
    g, d = gradient(1, N, K, seed=20, kind="strong"), gradient(1, N, K, seed=21)
    run = lambda x: mx.muon_update(cuda(x.astype(np.float32)), steps=1).float().cpu().numpy().astype(np.float64)  # noqa: E731
    assert np.array_equal(run(-g), -run(g))
    t = 0.25
    got, want = run(g + t * d) - run(g - t * d), muon(g + t * d, steps=1)[0] - muon(g - t * d, steps=1)[0]
    # each side is off by at most REL of its norm, the outputs' norms are alike
    assert np.linalg.norm(got - want) <= 2 * REL * np.linalg.norm(muon(g, steps=1)[0])


def test_large_sampled():
    """One full-size tall matrix against the iteration in 64 bits on the GPU."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(11)
    g = (torch.randn(2, 2048, 1408, generator=gen, device="cuda") * 1e-3).bfloat16()
    out = mx.muon_update(g).double()
    for e in range(2):
        X = g[e].double().T
        X /= X.norm() + 1e-7
        for _ in range(5):
            A = X @ X.T
            X = 3.4445 * X + (-4.775 * A + 2.0315 * (A @ A)) @ X
        assert float((out[e] - X.T).norm() / X.norm()) < REL


def test_workspace_stream_and_graph():
    g, m0 = gradient(3, 150, 264, seed=12), gradient(3, 150, 264, seed=13)
    ref = mx.muon_update(cuda(g), cuda(m0))
    torch.cuda.synchronize()
    ws = torch.full((mx.muon_update_workspace_bytes(3, 150, 264),), 0xFF, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    gd, md, start = cuda(g), cuda(m0), cuda(m0)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = mx.muon_update(gd, md, workspace=ws)
    side.synchronize()
    assert torch.equal(got, ref)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(ref)
    with torch.cuda.graph(graph, stream=side):
        mx.muon_update(gd, md, out=out, workspace=ws)
    for _ in range(2):
        md.copy_(start)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    assert mx.device_status(clear=True) == 0


def test_two_streams_at_once():
    g = cuda(gradient(4, 600, 520, seed=14))
    ref = mx.muon_update(g)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for rep in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(mx.muon_update(g))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    assert mx.device_status(clear=True) == 0


def test_refusals():
    g = torch.zeros(2, 16, 24, device="cuda")
    with pytest.raises(TypeError):
        mx.muon_update(g.half())
    with pytest.raises(TypeError):
        mx.muon_update([1, 2])
    with pytest.raises(ValueError):
        mx.muon_update(g.cpu())
    with pytest.raises(ValueError):
        mx.muon_update(g[0, 0])
    with pytest.raises(ValueError):
        mx.muon_update(g.mT)
    with pytest.raises(TypeError):
        mx.muon_update(g, g.bfloat16())
    with pytest.raises(ValueError):
        mx.muon_update(g, torch.zeros(2, 24, 16, device="cuda"))
    with pytest.raises(ValueError):
        mx.muon_update(g, out=torch.empty(2, 24, 16, dtype=torch.bfloat16, device="cuda"))
    for kw in (dict(steps=0), dict(steps=17), dict(coeffs=(float("nan"), 0, 0)), dict(coeffs=(20.0, 0, 0)), dict(eps=-1.0),
               dict(mu=float("inf"))):
        with pytest.raises(mx.Mxfp8Error) as e:
            mx.muon_update(g, **kw)
        assert e.value.code == -1
    with pytest.raises(mx.Mxfp8Error) as e:
        mx.muon_update(torch.zeros(2, 16, 20, device="cuda"))  # K % 8
    assert e.value.code == -2
    with pytest.raises(mx.Mxfp8Error) as e:
        mx.muon_update(g, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.code == -5
    assert mx.muon_update(torch.zeros(0, 16, 24, device="cuda")).shape == (0, 16, 24)
    torch.cuda.synchronize()
    assert mx.device_status(clear=True) == 0
