"""The expert-weight operators on planes of more than 2 and 4 GB, where byte and
element offsets pass 32 bits. A few matrices or experts, the last ones among
them, are checked in 64 bits on the GPU."""
import pytest
import torch

import moe_ragged_contraction_gb300 as mx
from _experts_ref import e4m3_table

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def room():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.build()
    mx.device_status(clear=True)
    yield
    torch.cuda.empty_cache()


def generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def test_layer_with_planes_over_4_gb():
    """320 experts of H = 4096, I = 2048: 5.4 GB of up/gate weights, 2.7 GB of down weights. Tolerance as in the layer's other tests."""
    T, H, I, E, k = 24, 4096, 2048, 320, 6
    gen = generator(1)

    def weights(rows, cols, shift):
        q = torch.randint(0, 0x60, (E, rows, cols), dtype=torch.uint8, device="cuda", generator=gen)  # magnitudes up to 30, no NaN
        q |= torch.randint(0, 2, (E, rows, cols), dtype=torch.uint8, device="cuda", generator=gen) << 7
        return q, torch.randint(shift, shift + 3, (E, rows, cols // 32), dtype=torch.uint8, device="cuda", generator=gen)

    w13, s13 = weights(2 * I, H, 117)
    w2, s2 = weights(H, I, 117)
    assert w13.numel() > 2 ** 32 and w2.numel() > 2 ** 31
    x = torch.randn(T, H, generator=gen, device="cuda").bfloat16()
    router = (torch.randn(E, H, generator=gen, device="cuda") / 64).bfloat16()
    bias = torch.zeros(E, device="cuda")
    bias[[0, 1, 127, 128, 318, 319]] = 2.0  # (softmax scores are at most one)
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    y = mx.moe_layer(x, router, w13, s13, w2, s2, k, bias=bias, topk_ids=ids, topk_weights=w)
    torch.cuda.synchronize()
    assert mx.device_status(clear=True) == 0
    assert sorted(set(ids.flatten().tolist())) == [0, 1, 127, 128, 318, 319]
    table = torch.from_numpy(e4m3_table()).cuda()
    decode = lambda q, s: table[q.int()] * torch.exp2(s.double() - 127).repeat_interleave(32, -1)  # noqa: E731
    want, acc = torch.zeros(T, H, dtype=torch.float64, device="cuda"), torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in (0, 1, 127, 128, 318, 319):
        we = (w * (ids == e)).sum(-1).double()
        gu = x.double() @ decode(w13[e], s13[e]).T
        h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
        d = decode(w2[e], s2[e])
        want += we[:, None] * (h @ d.T)
        acc += we[:, None] * (h.square() @ d.square().T).sqrt()
    assert bool((y.double() - want).abs().le(2.0 ** -9 * want.abs() + 6 * 2.0 ** -8 / 4 * acc).all())


def test_update_with_planes_over_4_gb():
    """130 matrices of 4096 x 4096: 2.2e9 elements, planes of 4.4 GB, momentum of 8.7 GB; two steps."""
    E, N = 130, 4096
    gen = generator(2)
    g = torch.empty(E, N, N, dtype=torch.bfloat16, device="cuda")
    m = torch.empty(E, N, N, device="cuda")
    for e in range(E):
        g[e] = torch.randn(N, N, generator=gen, device="cuda") * 1e-3
        m[e] = torch.randn(N, N, generator=gen, device="cuda") * 1e-3
    which = (0, 63, 64, 127, 128, 129)  # about elements 2^30 and 2^31 too
    old = {e: m[e].clone() for e in which}
    out = mx.muon_update(g, m, steps=2)
    torch.cuda.synchronize()
    assert mx.device_status(clear=True) == 0
    for e in which:
        m1 = 0.95 * old[e].double() + g[e].double()
        assert torch.allclose(m[e].double(), m1, rtol=2e-6, atol=1e-9)
        X = g[e].double() + 0.95 * m1
        X /= X.norm() + 1e-7
        for _ in range(2):
            A = X @ X.T
            X = 3.4445 * X + (-4.7750 * A + 2.0315 * (A @ A)) @ X
        assert float((out[e].double() - X).norm() / X.norm()) <= 4.5e-3, e  # (as in the update's other tests)


def test_small_updates_over_2_gb():
    """2048 matrices of 128 x 2048, one cluster each: the same bits as in a call of their own."""
    E = 2048
    gen = generator(3)
    g = torch.randn(E, 128, 2048, generator=gen, device="cuda")
    assert g.numel() * 4 > 2 ** 31 - 1
    out = mx.muon_update(g)
    for e in (0, 1023, 1024, 2047):
        assert torch.equal(out[e], mx.muon_update(g[e]))
    assert mx.device_status(clear=True) == 0
