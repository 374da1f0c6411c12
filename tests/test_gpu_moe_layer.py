"""The expert layer for a few tokens (moe_layer) against a 64-bit implementation
on the host: sizes that fill no tile, every token count class, both scores,
bias, renormalisation, experts that live elsewhere, ties, NaN, streams, CUDA
graphs, and the refusals.

Tolerance (derived, not fitted). The output is rounded to bf16: relative error
at most 2^-9 of the value. Before that the only rounding coarser than fp32 is
that of the inner activations h to two E4M3 pieces. The first piece leaves at
most 2^-4 |h| (half a unit of 4 significant bits), the second at most 2^-4 of
that, 2^-8 |h|; or, for values far below their 32-block's largest, half the
subnormal step of the second piece, 2^-10 / 448 * 2 of that piece's largest,
which is below 2^-22 of the block's largest. Each output sums I independent
such errors: at 2^-8 for each and random signs, 2^-8 sqrt(sum (w W2 h)^2), of
which six standard deviations are never exceeded in these tests (the errors are
in fact about four times smaller than 2^-8 on average). With fp32 sums of up
to a few thousand products on top (2^-20 of the same root sum): tol = 2^-9 |y| + 6 * 2^-8 / 4 * acc.
"""
import numpy as np
import pytest
import torch

import moe_ragged_contraction_gb300 as mx
import oracle
from _experts_ref import bf16_round, choice_values, dequantise, moe_layer as ref_layer, route

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.build()
    oracle.build()
    mx.load()
    mx.device_status(clear=True)


def make(T, H, I, experts, local, seed, spread=1.5):
    rng = np.random.default_rng(seed)
    x = bf16_round(rng.standard_normal((T, H)) * np.exp(rng.standard_normal((1, H))))
    router = bf16_round(rng.standard_normal((experts, H)) * spread / np.sqrt(np.square(x).sum(-1).mean() if T else H))
    def weights(rows, cols):
        w = (rng.standard_normal((local * rows, cols)) * np.exp(rng.standard_normal((local * rows, 1)) * 0.5) / np.sqrt(cols)).astype(np.float32)
        q, s = oracle.quantize_tokenwise(w)
        return q.reshape(local, rows, cols), s.reshape(local, rows, cols // 32)
    w13, s13 = weights(2 * I, H)
    w2, s2 = weights(H, I)
    return x, router, w13, s13, w2, s2


def cuda(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t.to(dtype) if dtype else t


def device_args(x, router, w13, s13, w2, s2):
    return cuda(x, torch.bfloat16), cuda(router, torch.bfloat16), cuda(w13), cuda(s13), cuda(w2), cuda(s2)


def check(x, router, w13, s13, w2, s2, top_k, got, ids, weights, first=0, **kw):
    rid, rw, gap = route(x, router, top_k, **kw)
    clear = gap > 1e-5  # far enough from a tie for the fp32 logits to decide as the 64-bit ones
    ids, weights = ids.cpu().numpy(), weights.cpu().numpy()
    assert clear.any() and np.array_equal(ids[clear], rid[clear])
    # nearer a tie: other experts, or another order, but of values as large
    _, choice = choice_values(x, router, kw.get("bias"), kw.get("score", "softmax"))
    assert all(len(set(row)) == top_k for row in ids.tolist())
    assert np.allclose(np.take_along_axis(choice, ids, 1), np.take_along_axis(choice, rid, 1), rtol=0, atol=1e-5)
    assert np.allclose(weights[clear], rw[clear], rtol=2e-5, atol=1e-7)
    # the experts' products with the routing that was taken
    y, acc = ref_layer(x, dequantise(w13, s13), dequantise(w2, s2), ids, weights.astype(np.float64), first)
    g = got.float().cpu().numpy().astype(np.float64)
    tol = 2.0 ** -9 * np.abs(y) + 6 * 2.0 ** -8 / 4 * acc
    assert np.all(np.abs(g - y) <= tol), float(np.max(np.abs(g - y) - tol))
    return rid


def run(args, top_k, **kw):
    T = args[0].shape[0]
    ids = torch.full((T, top_k), -1, dtype=torch.int32, device="cuda")
    weights = torch.full((T, top_k), float("nan"), dtype=torch.float32, device="cuda")
    out = torch.full(args[0].shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    r = mx.moe_layer(*args, top_k, out=out, topk_ids=ids, topk_weights=weights, **kw)
    assert r is out
    torch.cuda.synchronize()
    assert mx.device_status(clear=True) == 0
    return out, ids, weights


@pytest.mark.parametrize("T,H,I,experts,local,first,top_k,score,renorm,scale,bias", [
    (1, 32, 32, 1, 1, 0, 1, "softmax", True, 1.0, False),        # the smallest sizes: one partial K-step each way
    (1, 256, 128, 4, 4, 0, 2, "softmax", True, 1.0, False),
    (1, 2048, 1408, 16, 16, 0, 6, "softmax", False, 1.0, False),
    (2, 96, 160, 5, 3, 1, 2, "sigmoid", False, 2.5, True),       # tiles cut inside, scale rows of 3 and 5 bytes
    (3, 1056, 352, 21, 13, 4, 3, "sigmoid", True, 1.0, True),
    (8, 640, 416, 32, 32, 0, 8, "softmax", True, 1.0, False),    # the last size where every CTA routes for itself
    (9, 640, 416, 32, 32, 0, 8, "softmax", True, 1.0, False),    # the first where tokens are shared out
    (16, 512, 96, 40, 10, 30, 4, "sigmoid", True, 2.5, True),    # 16 tokens: the narrow router tile, its last size
    (17, 512, 96, 40, 10, 30, 4, "sigmoid", True, 2.5, True),
    (33, 224, 288, 3, 3, 0, 3, "softmax", True, 1.0, False),     # every token to every expert
    (64, 288, 64, 130, 97, 20, 7, "sigmoid", False, 1.0, True),
    (65, 160, 224, 2, 2, 0, 2, "softmax", True, 1.0, False),     # more than 128 columns (two scale blocks), one accumulator
    (128, 384, 192, 2, 1, 1, 1, "softmax", False, 1.0, False),   # up to 256 columns: the widest MMA, the shortest ring
    (128, 320, 160, 1, 1, 0, 1, "sigmoid", True, 1.0, False),    # all 128 tokens to the only expert
    (100, 96, 96, 1024, 700, 200, 16, "softmax", True, 1.0, True),  # the most experts and the largest top-k
])
def test_against_64_bits(T, H, I, experts, local, first, top_k, score, renorm, scale, bias):
    ops = make(T, H, I, experts, local, seed=T * 1000 + H + I)
    b = np.random.default_rng(7).standard_normal(experts).astype(np.float32) * 0.05 if bias else None
    args = device_args(*ops)
    kw = dict(score=score, renormalize=renorm, scale=scale)
    out, ids, weights = run(args, top_k, bias=None if b is None else cuda(b), first_expert=first, **kw)
    check(*ops, top_k, out, ids, weights, first=first, bias=b, **kw)
    again, ids2, weights2 = run(args, top_k, bias=None if b is None else cuda(b), first_expert=first, **kw)
    assert torch.equal(out, again) and torch.equal(ids, ids2) and torch.equal(weights, weights2)


def test_tokens_without_local_experts_are_exact_zeros():
    x, router, w13, s13, w2, s2 = make(12, 128, 64, 8, 2, seed=5)
    x[:, 0] = 4.0
    router[:, 0] = 0.0
    router[2:5, 0] = 8.0  # experts 2, 3, 4 win everywhere; 6 and 7 live here
    args = device_args(x, router, w13, s13, w2, s2)
    out, ids, _ = run(args, 3, first_expert=6)
    assert set(ids.cpu().numpy().ravel()) == {2, 3, 4}
    assert not out.view(torch.int16).any()


def test_ties_go_to_the_lower_expert_and_nan_counts_as_lowest():
    x, router, w13, s13, w2, s2 = make(3, 64, 32, 70, 70, seed=6)
    router[:] = router[:1]       # every expert the same logit
    args = device_args(x, router, w13, s13, w2, s2)
    _, ids, _ = run(args, 5)
    assert np.array_equal(ids.cpu().numpy(), np.tile(np.arange(5, dtype=np.int32), (3, 1)))
    bias = torch.zeros(70, device="cuda")
    bias[[3, 40, 69]] = 1.0
    bias[0] = float("nan")
    _, ids, _ = run(args, 5, bias=bias)
    assert np.array_equal(ids.cpu().numpy(), np.tile(np.array([3, 40, 69, 1, 2], np.int32), (3, 1)))


def test_nan_token_and_nan_weights_stay_apart():
    x, router, w13, s13, w2, s2 = make(6, 256, 128, 4, 4, seed=8)
    args = list(device_args(x, router, w13, s13, w2, s2))
    clean, ids, _ = run(args, 2)
    args[0] = args[0].clone()
    args[0][2, 17] = float("nan")
    args[0][4, 200] = float("inf")
    out, _, _ = run(args, 2)
    keep = [0, 1, 3, 5]
    assert torch.equal(out[keep], clean[keep])
    assert torch.isnan(out[2]).all() and torch.isnan(out[4]).all()
    # a NaN scale in a down row: that column of the tokens that use the expert
    args[0] = cuda(x, torch.bfloat16)
    s2n = args[5].clone()
    e = int(ids[0, 0])
    s2n[e, 9, 1] = 255
    args[5] = s2n
    out, _, _ = run(args, 2)
    hit = (ids == e).any(1)
    assert torch.isnan(out[hit][:, 9]).all() and not torch.isnan(out[~hit]).any()
    rest = torch.ones(256, dtype=torch.bool)
    rest[9] = False
    assert torch.equal(out[:, rest], clean[:, rest])


def test_wide_range_of_activations():
    """Values spread over 2^-30 .. 2^12 inside blocks, zero blocks, a zero token: the pieces keep what matters."""
    x, router, w13, s13, w2, s2 = make(5, 512, 256, 3, 3, seed=9)
    rng = np.random.default_rng(10)
    x = bf16_round(x * np.exp2(rng.integers(-30, 13, x.shape)).astype(np.float32))
    x[:, 64:128] = 0
    x[3] = 0
    router *= np.float32(1e-3)
    router = bf16_round(router)
    args = device_args(x, router, w13, s13, w2, s2)
    out, ids, weights = run(args, 3)
    y, acc = ref_layer(x, dequantise(w13, s13), dequantise(w2, s2), ids.cpu().numpy(), weights.cpu().numpy().astype(np.float64))
    g = out.float().cpu().numpy()
    assert np.all(np.abs(g - y) <= 2.0 ** -9 * np.abs(y) + 6 * 2.0 ** -8 / 4 * acc)
    assert not out[3].any()


def test_workspace_stream_and_graph():
    T, H, I, E, k = 11, 384, 224, 9, 3
    ops = make(T, H, I, E, E, seed=12)
    args = device_args(*ops)
    ref, _, _ = run(args, k)
    need = mx.moe_layer_workspace_bytes(T, E, E, H, I, k)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")  # whatever the scratch holds
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = mx.moe_layer(*args, k, workspace=ws)
    side.synchronize()
    assert torch.equal(got, ref)
    got2 = mx.moe_layer(*args, k, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(got2, ref)
    g = torch.cuda.CUDAGraph()
    out = torch.empty_like(ref)
    with torch.cuda.graph(g, stream=side):
        mx.moe_layer(*args, k, out=out, workspace=ws)
    x2 = cuda(bf16_round(np.random.default_rng(3).standard_normal((T, H))), torch.bfloat16)
    want, _, _ = run([x2, *args[1:]], k)
    args[0].copy_(x2)  # a replay reads the buffers anew
    out.zero_()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert mx.device_status(clear=True) == 0


def test_two_streams_at_once():
    """Calls on two streams, each with its own scratch, overlap on the device without waiting on each other."""
    ops = make(20, 1024, 512, 24, 24, seed=13)
    args = device_args(*ops)
    ref, _, _ = run(args, 4)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for rep in range(8):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(mx.moe_layer(*args, 4))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    assert mx.device_status(clear=True) == 0


def test_few_long_tiles_are_cut_into_parts():
    """One chosen expert with few, long tiles: parts along both contractions, summed in order."""
    for T, H, I in ((1, 2048, 64), (3, 96, 2048), (2, 1312, 800)):
        ops = make(T, H, I, 6, 2, seed=H + I)
        args = device_args(*ops)
        bias = torch.tensor([0, 0, 9.0, 0, 0, 0], device="cuda")
        out, ids, weights = run(args, 2, bias=bias, first_expert=2)
        check(*ops, 2, out, ids, weights, first=2, bias=bias.cpu().numpy())
        again, _, _ = run(args, 2, bias=bias, first_expert=2)
        assert torch.equal(out, again)


@pytest.mark.parametrize("T,H,I", [
    (1, 7168, 64), (40, 4512, 160),        # long rows of x: the up and gate products in parts
    (3, 96, 4128), (17, 288, 4096),        # long rows of h: the down products in parts
    (1, 4128, 4224), (128, 4096, 32),      # both; the most tokens
])
def test_long_contractions_are_cut_into_parts(T, H, I):
    """Few tiles with contractions of 4096 columns and more, odd numbers of K-steps among them, two experts of six here."""
    ops = make(T, H, I, 6, 2, seed=H + I)
    args = device_args(*ops)
    out, ids, weights = run(args, 3, first_expert=2)
    check(*ops, 3, out, ids, weights, first=2)
    again, _, _ = run(args, 3, first_expert=2)
    assert torch.equal(out, again)


@pytest.mark.parametrize("H,I", [(1056, 32), (64, 1056)])
def test_largest_lists_and_fewest_stages(H, I):
    """The most tokens, experts and choices, every token with the same sixteen experts: 256 columns, three stages."""
    T, experts, top_k = 128, 1024, 16
    x, router, w13, s13, w2, s2 = make(T, H, I, experts, experts, seed=77)
    bias = np.zeros(experts, np.float32)
    bias[np.arange(top_k) * 63 + 5] = 2.0  # (softmax scores are at most one)
    args = device_args(x, router, w13, s13, w2, s2)
    out, ids, weights = run(args, top_k, bias=cuda(bias))
    check(x, router, w13, s13, w2, s2, top_k, out, ids, weights, bias=bias)
    assert set(ids.cpu().numpy().ravel().tolist()) == set((np.arange(top_k) * 63 + 5).tolist())


def test_example_runs():
    """The example's path: gradients, update, quantised weights, layer; an expert without tokens stays as it was."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_step.py")
    spec = importlib.util.spec_from_file_location("expert_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    before, after, moms, update = m.main(E=4, H=256, I=128, tokens_per_expert=64, steps=2)
    assert torch.isfinite(after).all() and not torch.equal(before, after)
    assert not update[2].any() and not moms[1][2].any() and update[1].any()


def test_scale_planes_off_by_a_word():
    """Scale planes are 4-byte aligned, no more, also where their rows are whole 8-byte words."""
    T, H, I, experts = 3, 512, 256, 4
    x, router, w13, s13, w2, s2 = make(T, H, I, experts, experts, 31)
    args = list(device_args(x, router, w13, s13, w2, s2))
    want = run(args, 2)[0]
    for i in (3, 5):
        room = torch.zeros(args[i].numel() + 4, dtype=torch.uint8, device="cuda")
        off = room[4:].view(args[i].shape)
        off.copy_(args[i])
        assert off.data_ptr() % 8 == 4
        args[i] = off
    assert torch.equal(run(args, 2)[0], want)


def test_no_tokens():
    ops = make(1, 64, 32, 4, 4, seed=14)
    args = list(device_args(*ops))
    args[0] = args[0][:0]
    assert mx.moe_layer(*args, 2).shape == (0, 64)


def test_refusals():
    ops = make(4, 64, 32, 4, 4, seed=15)
    a = device_args(*ops)
    ok = dict(x=a[0], router=a[1], w13=a[2], s13=a[3], w2=a[4], s2=a[5], top_k=2)
    with pytest.raises(TypeError):
        mx.moe_layer(**{**ok, "x": a[0].float()})
    with pytest.raises(TypeError):
        mx.moe_layer(**{**ok, "x": ops[0]})
    with pytest.raises(ValueError):
        mx.moe_layer(**{**ok, "x": a[0].cpu()})
    with pytest.raises(ValueError):
        mx.moe_layer(**{**ok, "router": torch.cat([a[1], a[1]], 1)[:, ::2]})  # not contiguous
    with pytest.raises(ValueError):
        mx.moe_layer(**{**ok, "s13": a[3][:, :-1].contiguous()})
    with pytest.raises(ValueError):
        mx.moe_layer(**{**ok, "w2": a[4][:3].contiguous()})
    with pytest.raises(ValueError):
        mx.moe_layer(**ok, score="tanh")
    with pytest.raises(ValueError):
        mx.moe_layer(**ok, out=torch.empty(4, 32, dtype=torch.bfloat16, device="cuda"))
    for kw in (dict(top_k=5), dict(top_k=0), dict(first_expert=1), dict(first_expert=-1), dict(scale=float("nan"))):
        with pytest.raises(mx.Mxfp8Error) as e:
            mx.moe_layer(**{**ok, **kw})
        assert e.value.code == -1
    with pytest.raises(mx.Mxfp8Error):
        mx.moe_layer(**{**ok, "x": torch.zeros(129, 64, dtype=torch.bfloat16, device="cuda")})
    with pytest.raises(mx.Mxfp8Error) as e:
        mx.moe_layer(**ok, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.code == -5
    torch.cuda.synchronize()
    assert mx.device_status(clear=True) == 0
