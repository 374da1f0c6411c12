"""The operators of a training step together, as a step uses them: bit for bit where every product and sum is exact, the
layer of the example against its 64-bit gradients, one captured step replayed, and outputs that belong to the stream."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import moe_ragged_contraction_gb300 as mx
from moe_ragged_contraction_gb300 import _lib
import _experts_ref as X
import _step_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib_built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.build()
    yield
    assert mx.device_status(clear=True) == 0


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def rounded(a):
    """64-bit values as bf16 bit patterns (zeros without their sign)."""
    b = X.bf16_round(a).view(np.uint32) >> 16
    return np.where(b == 0x8000, 0, b).astype(np.uint16)


def bits(t):
    b = t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
    return np.where(b == 0x8000, 0, b)


@pytest.mark.parametrize("T,k,E,first,local,H,N", [(600, 3, 5, 0, 5, 256, 128), (257, 2, 24, 8, 8, 512, 64), (1, 1, 4, 0, 4, 128, 32), (40, 2, 6, 2, 2, 96, 96)])
def test_linear_layer_bit_for_bit(T, k, E, first, local, H, N):
    """A linear expert layer on small integers and weights that are powers of two: all quantisation, products and sums are
    exact, and each result is the exact value rounded to bf16 once."""
    rng = np.random.default_rng(T + E)
    sparse = lambda shape, p: rng.choice([-1.0, 1.0], shape) * (rng.random(shape) < p)  # noqa: E731
    x, W, dout = sparse((T, H), 0.2), sparse((local, N, H), 0.3), rng.choice([-2.0, -1.0, 0.0, 1.0, 2.0], (T, N))
    w = rng.choice([0.25, 0.5, 1.0, 2.0], (T, k))
    ids = rng.integers(0, E, (T, k))
    ids[T - T // 10:] = -1
    plan = mx.token_plan(dev(ids), local, first_expert=first)
    rows = plan.src.numel()
    offs, slot, src, _ = R.plan(ids, first, local, 32, rows)
    assert np.array_equal(plan.slot.cpu().numpy(), slot)
    bf = lambda a: dev(a.astype(np.float32)).bfloat16()  # noqa: E731

    def quant(a):
        q, s = mx.quantize_tokenwise(a.float().reshape(-1, a.shape[-1]).contiguous())
        return q.view(a.shape), s.view(*a.shape[:-1], -1)

    y = mx.grouped_gemm(*mx.token_dispatch_mxfp8(bf(x), plan), *quant(dev(W)), plan.offs)
    out = mx.token_combine(y, dev(w.astype(np.float32)), plan)
    dy, dw = mx.token_combine_grad(bf(dout), y, dev(w.astype(np.float32)), plan)
    dxs = mx.grouped_gemm(*quant(dy), *quant(dev(np.ascontiguousarray(W.transpose(0, 2, 1)))), plan.offs)
    dx = mx.token_dispatch_grad(dxs, plan)
    dW = mx.wgrad_grouped(*mx.quantize_transpose_bf16(dy), *mx.quantize_transpose_bf16(mx.token_dispatch(bf(x), plan)), plan.offs)

    xs = R.dispatch(x, src, k)
    start = np.concatenate(([0], offs[:-1]))
    ry = np.zeros((rows, N))
    for e in range(local):
        ry[start[e]:offs[e]] = xs[start[e]:offs[e]] @ W[e].T
    ry = X.bf16_round(ry).astype(np.float64)
    assert np.array_equal(bits(y), rounded(ry))
    assert np.array_equal(bits(out), rounded(R.combine(ry, w, slot)[0]))
    rdy, rdw, _ = R.combine_grad(dout, ry, w, slot, rows)
    assert np.array_equal(bits(dy), rounded(rdy)) and np.array_equal(dw.double().cpu().numpy(), rdw)
    rdxs, rdW = np.zeros((rows, H)), np.zeros((local, N, H))
    for e in range(local):
        rdxs[start[e]:offs[e]] = rdy[start[e]:offs[e]] @ W[e]
        rdW[e] = rdy[start[e]:offs[e]].T @ xs[start[e]:offs[e]]
    rdxs = X.bf16_round(rdxs).astype(np.float64)
    assert np.array_equal(bits(dx), rounded(R.combine(rdxs, None, slot)[0]))
    assert np.array_equal(bits(dW), rounded(rdW))

    # the gradients clipped and updated: the norm of what was written, the update as of the scaled gradient
    norm = mx.clip_grads([dW, dw], 0.5)
    want = R.norm([X.bf16_round(rdW).astype(np.float64), rdw])
    assert abs(float(norm) - want) <= 1e-6 * want + 1e-30
    update = mx.muon_update(dW)
    assert torch.isfinite(update).all() and bool(update.any()) == bool(rdW.any())


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "layer_step.py")
    spec = importlib.util.spec_from_file_location("layer_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_runs():
    out, norms = example().main(T=200, E=4, H=256, I=128, steps=2)
    assert torch.isfinite(out).all() and all(torch.isfinite(n) for n in norms)


def test_example_gradients():
    """Against the layer's gradients in 64 bits, weights as quantised. An operand quantised to E4M3 is off by at most 2^-4
    of its elements, so by at most 2^-4 of its norm: x enters g and u, h and dy and dgu once each more. Random products carry such
    an error on in proportion; the factor of one quarter is the sum of four of them. (A mistake in the wiring gives 1 and more.)"""
    m = example()
    T, E, H, I, k = 300, 4, 256, 128, 2
    gen = torch.Generator(device="cuda")
    gen.manual_seed(9)
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731

    def decoded(w):
        q, s = m.quantised(w)
        return dev(X.dequantise(q.cpu().numpy(), s.cpu().numpy())).requires_grad_()

    w13, w2, router = rand(E, 2 * I, H) / 16, rand(E, H, I) / 11, rand(E, H) / 16
    x, dout = rand(T, H).bfloat16(), rand(T, H).bfloat16()
    out, dx, (dw13, dw2, drouter) = m.layer(x, dout, router, w13, w2, k)
    X64, r64, a13, a2 = x.double().requires_grad_(), router.double().requires_grad_(), decoded(w13), decoded(w2)
    score, ids = torch.topk(X64.detach() @ r64.T, k)
    p = torch.softmax(score, -1)
    gu = torch.einsum("th,tkih->tki", X64, a13[ids])
    h = torch.nn.functional.silu(gu[..., :I]) * gu[..., I:]
    ref = torch.einsum("tk,tki,tkhi->th", p, h, a2[ids])
    grads = torch.autograd.grad(ref, (X64, a13, a2, r64), dout.double())
    for got, want in zip((out, dx, dw13, dw2, drouter), (ref, *grads)):
        assert float((got.double() - want.detach()).norm() / want.detach().norm()) < 0.25


def test_a_captured_step():
    """The whole layer in one graph, replayed on other tokens with another routing."""
    T, k, E, H, N = 333, 2, 6, 128, 64
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    q, s = mx.quantize_tokenwise(rand(E * N, H))
    qt, st = mx.quantize_tokenwise(rand(E * H, N))
    sets = [(rand(T, H).bfloat16(), rand(T, N).bfloat16(), torch.randint(-1, E, (T, k), generator=gen, device="cuda"), torch.rand((T, k), generator=gen, device="cuda")) for _ in range(3)]
    rows = mx.token_plan_rows(T, k, E)
    ws = torch.empty(mx.workspace_bytes(E, N, H, rows), dtype=torch.uint8, device="cuda")
    gws = torch.empty(mx.grad_workspace_bytes(2), dtype=torch.uint8, device="cuda")

    def step(x, dout, ids, w):
        plan = mx.token_plan(ids, E)
        y = mx.grouped_gemm(*mx.token_dispatch_mxfp8(x, plan), q.view(E, N, H), s.view(E, N, -1), plan.offs)
        out = mx.token_combine(y, w, plan)
        dy, dw = mx.token_combine_grad(dout, y, w, plan)
        dx = mx.token_dispatch_grad(mx.token_dispatch(x, plan), plan)
        dW = mx.wgrad_grouped(*mx.quantize_transpose_bf16(dy), *mx.quantize_transpose_bf16(mx.token_dispatch(x, plan)), plan.offs, workspace=ws)
        before = dW.clone()
        norm = mx.clip_grads([dW, dw], 1.0, workspace=gws)
        return [*plan, out, dy, dx, before, dW, dw, norm]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        want = [step(*a) for a in sets]
    torch.cuda.synchronize()
    live = [a.clone() for a in sets[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):  # (grouped_gemm's scratch is the stream's)
        got = step(*live)
    for i in (1, 2, 0, 1):
        for a, b in zip(live, sets[i]):
            a.copy_(b)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want[i]):
            assert torch.equal(a, b)


def test_threads_on_streams_of_their_own():
    """Four host threads at once, each with its stream and its routing."""
    import threading

    T, k, E, H = 900, 4, 24, 512
    gen = torch.Generator(device="cuda")
    gen.manual_seed(21)

    def chain(a, stream):
        ids, x, w, grads = a
        plan = mx.token_plan(ids, E, stream=stream)
        xs = mx.token_dispatch(x, plan, stream=stream)
        out = mx.token_combine(xs, w, plan, stream=stream)
        dy, dw = mx.token_combine_grad(out, xs, w, plan, stream=stream)
        clipped = [torch.zeros_like(g) for g in grads]
        stream.wait_stream(torch.cuda.current_stream())
        norm = mx.clip_grads(grads, 1.0, out=clipped, stream=stream)
        return [*plan, xs, out, dy, dw, norm, *clipped]

    sets = [(torch.randint(-1, E, (T, k), generator=gen, device="cuda"), torch.randn((T, H), generator=gen, device="cuda").bfloat16(), torch.rand((T, k), generator=gen, device="cuda"),
             [torch.randn(n, generator=gen, device="cuda") * (i + 1) for n in (70001, 33)]) for i in range(4)]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    want = [chain(a, s) for a, s in zip(sets, streams)]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def work(i):
        try:
            for _ in range(30):
                got[i] = chain(sets[i], streams[i])
            streams[i].synchronize()
        except Exception as e:  # noqa: BLE001 (reported below)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for g, e in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, e))


def test_scratch_under_capture():
    """Clipping on a stream without scratch, captured: refused with a message, nothing recorded; the token operators need none."""
    g = [torch.ones(100, device="cuda")]
    ids = torch.zeros((4, 1), dtype=torch.int32, device="cuda")
    mx.token_plan(ids, 2)
    mx.grad_norm(g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        plan = mx.token_plan(ids, 2)
        with pytest.raises(mx.Mxfp8Error) as e:
            mx.grad_norm(g)
        assert e.value.code == _lib.ENOWS
    graph.replay()
    torch.cuda.synchronize()
    assert plan.slot.view(-1).tolist() == [0, 1, 2, 3]


def calls(t):
    """name -> call(stream=...) returning the outputs it allocates."""
    bf, f32, i32, i64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
    T, k, H, rows = 6, 2, 64, 64
    plan = mx.TokenPlan(t(i32, 3), t(i32, T, k), t(i32, rows))
    x, y, w = t(bf, T, H), t(bf, rows, H), t(f32, T, k)
    return {
        "token_plan": lambda stream: list(mx.token_plan(t(i64, T, k), 3, stream=stream)),
        "token_dispatch": lambda stream: [mx.token_dispatch(x, plan, stream=stream)],
        "token_dispatch_mxfp8": lambda stream: list(mx.token_dispatch_mxfp8(x, plan, stream=stream)),
        "token_dispatch_grad": lambda stream: [mx.token_dispatch_grad(y, plan, stream=stream)],
        "token_combine": lambda stream: [mx.token_combine(y, w, plan, stream=stream)],
        "token_combine_grad": lambda stream: list(mx.token_combine_grad(x, y, w, plan, stream=stream)),
        "grad_norm": lambda stream: [mx.grad_norm([y, w], stream=stream)],
        "clip_grads": lambda stream: [mx.clip_grads([y, w], 1.0, stream=stream)],
    }


@pytest.mark.parametrize("name", ["token_plan", "token_dispatch", "token_dispatch_mxfp8", "token_dispatch_grad", "token_combine", "token_combine_grad", "grad_norm", "clip_grads"])
def test_outputs_belong_to_the_stream(name):
    run = calls(lambda dtype, *shape: torch.zeros(shape, dtype=dtype, device="cuda"))[name]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream, want in ((side, side.cuda_stream), (None, torch.cuda.current_stream().cuda_stream)):
        outs = run(stream)
        torch.cuda.synchronize()
        segments = torch.cuda.memory_snapshot()
        for o in outs:
            p = o.data_ptr()
            assert [s["stream"] for s in segments if s["address"] <= p < s["address"] + s["total_size"]] == [want]
