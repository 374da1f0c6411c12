"""Host-side checks of the expert-weight operators' C ABI (no GPU) and of the
64-bit implementations that the GPU tests compare with."""
import numpy as np
import pytest

import moe_ragged_contraction_gb300 as mx
from moe_ragged_contraction_gb300 import _lib
import _experts_ref as R

P = 0x10000  # 256-byte aligned fake address: never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    mx.build()
    return mx.load()


def moe(lib, x=P, T=4, router=P, bias=None, w13=P, s13=P, w2=P, s2=P, experts=8, first=0, local=8, H=64, I=32, top_k=2, score=0,
        renormalize=1, scale=1.0, out=P, ids=None, weights=None):
    return lib.mxfp8_moe_layer(x, T, router, bias, w13, s13, w2, s2, experts, first, local, H, I, top_k, score, renormalize, scale,
                               out, ids, weights, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), _lib.EINVAL), (dict(T=129), _lib.EINVAL), (dict(H=33), _lib.EINVAL), (dict(I=16), _lib.EINVAL),
    (dict(H=0), _lib.EINVAL), (dict(experts=0), _lib.EINVAL), (dict(experts=1025), _lib.EINVAL), (dict(local=0), _lib.EINVAL),
    (dict(first=1), _lib.EINVAL), (dict(first=-1), _lib.EINVAL), (dict(top_k=0), _lib.EINVAL), (dict(top_k=9), _lib.EINVAL),
    (dict(experts=64, top_k=17), _lib.EINVAL), (dict(score=2), _lib.EINVAL), (dict(scale=float("inf")), _lib.EINVAL),
    (dict(x=None), _lib.EINVAL), (dict(s2=None), _lib.EINVAL), (dict(out=None), _lib.EINVAL),
    (dict(x=P + 8), _lib.EALIGN), (dict(w13=P + 4), _lib.EALIGN), (dict(out=P + 2), _lib.EALIGN), (dict(s13=P + 2), _lib.EALIGN),
    (dict(bias=P + 1), _lib.EALIGN),
])
def test_moe_layer_host_validation(lib, kw, code):
    assert moe(lib, **kw) == code
    assert len(lib.mxfp8_last_error()) > 0


def test_moe_layer_no_tokens_is_noop(lib):
    assert moe(lib, T=0, x=None, out=None) == _lib.OK


def muon(lib, grad=P, gt=0, mom=None, E=2, N=16, K=24, mu=0.9, nesterov=1, steps=5, a=3.4, b=-4.7, c=2.0, eps=1e-7, out=P):
    return lib.mxfp8_muon_update(grad, gt, mom, E, N, K, mu, nesterov, steps, a, b, c, eps, out, None)


@pytest.mark.parametrize("kw,code", [
    (dict(E=-1), _lib.EINVAL), (dict(E=2049), _lib.EINVAL), (dict(N=0), _lib.EINVAL), (dict(K=0), _lib.EINVAL),
    (dict(N=32769), _lib.EINVAL), (dict(gt=2), _lib.EINVAL), (dict(steps=0), _lib.EINVAL), (dict(steps=17), _lib.EINVAL),
    (dict(a=float("nan")), _lib.EINVAL), (dict(c=17.0), _lib.EINVAL), (dict(eps=-1e-3), _lib.EINVAL),
    (dict(mu=float("inf")), _lib.EINVAL), (dict(K=20), _lib.EALIGN), (dict(grad=None), _lib.EINVAL), (dict(out=None), _lib.EINVAL),
    (dict(grad=P + 8), _lib.EALIGN), (dict(mom=P + 4), _lib.EALIGN),
])
def test_muon_update_host_validation(lib, kw, code):
    assert muon(lib, **kw) == code


def test_muon_update_no_matrices_is_noop(lib):
    assert muon(lib, E=0, grad=None, out=None) == _lib.OK


def test_workspace_bytes(lib):
    f = mx.moe_layer_workspace_bytes
    assert f(4, 8, 8, 64, 33, 2) == 0 and f(4, 8, 9, 64, 32, 2) == 0
    assert f(128, 64, 64, 2048, 1408, 6) > f(8, 64, 64, 2048, 1408, 6) > f(1, 64, 64, 2048, 1408, 6) > 0
    g = mx.muon_update_workspace_bytes
    assert g(1, 16, 20) == 0 and g(0, 16, 24) == 0
    # two planes of X twice, A and R: 8 bytes per element and 4 per element of the square
    assert g(8, 1408, 2048) >= 8 * (8 * 1408 * 2048 + 4 * 1408 * 1408)
    lib_ = mx.load()
    assert lib_.mxfp8_muon_update_ws(P, 0, None, 2, 16, 24, 0.9, 1, 5, 3.4, -4.7, 2.0, 1e-7, P, P, 16, None) == _lib.ENOWS
    assert lib_.mxfp8_muon_update_ws(P, 0, None, 2, 16, 24, 0.9, 1, 5, 3.4, -4.7, 2.0, 1e-7, P, P + 16, 1 << 30, None) == _lib.EALIGN


# ------------------------------------------------------------------ the 64-bit implementations

def test_reference_route_worked_example():
    x = np.array([[1.0, 0.0], [0.0, 2.0]], np.float32)
    router = np.array([[0.0, 0.0], [1.0, 1.0], [1.0, 0.5]], np.float32)
    ids, w, gap = R.route(x, router, 2, renormalize=True)
    assert ids.tolist() == [[1, 2], [1, 2]]  # the tie of the first token goes to the lower index
    assert np.allclose(w[0], 0.5) and np.allclose(w[1], np.exp([2, 1]) / np.exp([2, 1]).sum())
    assert gap[0] == 0


def test_reference_layer_is_the_dense_sum():
    rng = np.random.default_rng(0)
    x, w13, w2 = rng.standard_normal((3, 32)), rng.standard_normal((2, 8, 32)), rng.standard_normal((2, 32, 4))
    y, _ = R.moe_layer(x, w13, w2, np.array([[0, 1]] * 3), np.array([[1.0, 1.0]] * 3))
    gu = np.einsum("ekh,th->tek", w13, x)
    h = gu[..., :4] / (1 + np.exp(-gu[..., :4])) * gu[..., 4:]
    assert np.allclose(y, np.einsum("ehi,tei->th", w2, h))
    y2, _ = R.moe_layer(x, w13, w2, np.array([[5, 6]] * 3), np.array([[1.0, 1.0]] * 3), first=4)
    y1, _ = R.moe_layer(x, w13[1:], w2[1:], np.array([[0, 7]] * 3), np.array([[1.0, 1.0]] * 3))
    assert np.allclose(y2, y1)  # only expert 5 of [4, 6) is chosen and lives here


def test_reference_muon_acts_on_singular_values():
    """u = U S V^T goes to U p(p(... S / ||S||)) V^T with p(s) = a s + b s^3 + c s^5."""
    rng = np.random.default_rng(1)
    for shape in ((6, 9), (9, 6)):
        g = rng.standard_normal((1, *shape))
        U, S, V = np.linalg.svd(g[0], full_matrices=False)
        s = S / (np.linalg.norm(S) + 1e-7)
        for _ in range(5):
            s = 3.4445 * s - 4.7750 * s ** 3 + 2.0315 * s ** 5
        out, _ = R.muon(g)
        assert np.allclose(out[0], U * s @ V, atol=1e-9)


def test_reference_momentum():
    g, m = np.ones((1, 1, 1)), np.full((1, 1, 1), 2.0)
    _, m1 = R.muon(g, m, mu=0.5)
    assert m1[0, 0, 0] == 2.0  # 0.5 * 2 + 1


def test_split_of_bf16_into_two_e4m3_pieces_is_exact():
    """A bf16 value has 8 significant bits: its nearest E4M3 value leaves a remainder of at most 4."""
    table = R.e4m3_table()
    table = np.unique(table[np.isfinite(table)])
    v = np.array([(128 + f) * 2.0 ** (e - 7) for e in range(-5, 8) for f in range(128)])
    nearest = table[np.argmin(np.abs(table[None] - v[:, None]), 1)]
    rest = v - nearest
    scaled = rest * 2.0 ** 8  # the second piece has its own power-of-two scale
    assert np.abs(scaled[np.abs(v) < 2]).max() <= 448
    mant = np.abs(rest[rest != 0]) / 2.0 ** (np.floor(np.log2(np.abs(rest[rest != 0]))) - 3)
    assert np.all(mant == np.round(mant))  # at most 4 significant bits
