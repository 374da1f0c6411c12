"""Gradient norm and clipping on the GPU against 64 bits."""
import numpy as np
import pytest
import torch

import moe_ragged_contraction_gb300 as mx
from moe_ragged_contraction_gb300 import _lib
import _step_ref as R

pytestmark = pytest.mark.gpu

B16, F32 = torch.finfo(torch.bfloat16).eps / 2, torch.finfo(torch.float32).eps / 2
# a thread's sum: four chains of at most 16 fused steps and two sums (each off by F32 of a sum of positive terms), halved by
# the root; the root's rounding to fp32
NORM = (18 / 2 + 1) * F32 * 1.001
# the factor's rounding to fp32 and the product's, on top of the norm's error
FACTOR = (18 / 2 + 2) * F32 * 1.001


@pytest.fixture(scope="module", autouse=True)
def _lib_built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.build()
    yield
    assert mx.device_status(clear=True) == 0


def tensors(rng, sizes, kind="mixed", flat=False, scale=1.0):
    """Gradients of different strength; `flat`: views of one buffer a type, at whatever alignment comes."""
    types = {"bf16": [torch.bfloat16], "fp32": [torch.float32], "mixed": [torch.bfloat16, torch.float32, torch.bfloat16]}[kind]
    got, at = [], {}
    room = {t: torch.zeros(sum(sizes) + 64, dtype=t, device="cuda") for t in set(types)}
    for i, n in enumerate(sizes):
        t = types[i % len(types)]
        v = torch.from_numpy((rng.standard_normal(n) * scale * np.exp(rng.standard_normal())).astype(np.float32)).cuda().to(t)
        if flat:
            a = at.get(t, 1)
            room[t][a:a + n] = v
            v, at[t] = room[t][a:a + n], a + n
        got.append(v)
    return got


def np64(t):
    return t.double().cpu().numpy()


SIZES = [[1], [7], [8], [2049, 1, 0, 5], [16384, 16385, 3], [100003], [0, 0, 12], [513] * 64, [40, 1000] * 40, [33] * 1025, [1 << 20, 77, 3 * 10 ** 6 + 1]]


@pytest.mark.parametrize("flat", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp32", "mixed"])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_norm_and_clip(sizes, kind, flat):
    rng = np.random.default_rng(sum(sizes) + len(kind))
    g = tensors(rng, sizes, kind, flat)
    want = R.norm([np64(t) for t in g])
    got = float(mx.grad_norm(g))
    assert abs(got - want) <= NORM * want
    for max_norm in (want / 3, want * 3):
        c = R.factor(want, max_norm)
        before = [t.clone() for t in g]
        out = [torch.full_like(t, 5.0) for t in g]
        norm = mx.clip_grads(g, max_norm, out=out)
        assert norm.shape == () and float(norm) == got
        for t, b, o in zip(g, before, out):
            assert torch.equal(t, b)
            v = np64(b) * c
            rel = 0.0 if c == 1.0 else FACTOR + (B16 * 1.01 if b.dtype is torch.bfloat16 else 0.0)
            assert np.all(np.abs(np64(o) - v) <= rel * np.abs(v) + 2.0 ** -133)
        # in place (at the same addresses): the same bits
        assert float(mx.clip_grads(g, max_norm)) == got
        assert all(torch.equal(a, o) for a, o in zip(g, out))
        for t, b in zip(g, before):
            t.copy_(b)


@pytest.mark.parametrize("n,types", [(70000, "fp32"), (70000, "bf16"), (300, "fp32"), (9, "bf16")])
def test_flat_views_in_place(n, types):
    """Neighbours in one buffer, in place: each element is scaled once, and what lies between and around stays."""
    rng = np.random.default_rng(n)
    t = torch.bfloat16 if types == "bf16" else torch.float32
    flat = torch.from_numpy(rng.standard_normal(3 * n + 11).astype(np.float32)).cuda().to(t)
    before = flat.clone()
    views = [flat[1:n], flat[n:2 * n + 3], flat[2 * n + 5:3 * n + 4].view(-1, 1)]  # (a gap of two elements; the middle one touches the first)
    norm = mx.clip_grads(views, 0.5)
    want = R.norm([np64(before[1:n]), np64(before[n:2 * n + 3]), np64(before[2 * n + 5:3 * n + 4])])
    assert abs(float(norm) - want) <= NORM * want
    c = R.factor(want, 0.5)
    scaled = np64(before) * c
    untouched = np.zeros(flat.numel(), bool)
    untouched[0] = True
    untouched[2 * n + 3:2 * n + 5] = True
    untouched[3 * n + 4:] = True
    got = np64(flat)
    assert np.array_equal(got[untouched], np64(before)[untouched])
    rel = FACTOR + (B16 * 1.01 if types == "bf16" else 0.0)
    assert np.all(np.abs(got - scaled)[~untouched] <= rel * np.abs(scaled)[~untouched] + 2.0 ** -133)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("at", range(8))
@pytest.mark.parametrize("to", [0, 1, 3, 4])
def test_inputs_and_outputs_at_any_elements(kind, at, to):
    """Every distance of an output's address from its input's, modulo 16 bytes; nothing around the outputs is written."""
    rng = np.random.default_rng(8 * at + to)
    t = torch.bfloat16 if kind == "bf16" else torch.float32
    sizes = [50000, 3, 20001]
    src = torch.from_numpy(rng.standard_normal(80000).astype(np.float32)).cuda().to(t)
    dst = torch.full((80000,), 7.0, dtype=t, device="cuda")
    g = [src[at + o:at + o + n] for o, n in zip((0, 50000, 50010), sizes)]
    out = [dst[to + o:to + o + n] for o, n in zip((0, 50005, 50009), sizes)]
    norm = mx.clip_grads(g, 1.0, out=out)
    want = R.norm([np64(v) for v in g])
    assert abs(float(norm) - want) <= NORM * want
    rel = FACTOR + (B16 * 1.01 if kind == "bf16" else 0.0)
    touched = torch.zeros(80000, dtype=torch.bool, device="cuda")
    for a, b in zip(g, out):
        e = np64(a) * R.factor(want, 1.0)
        assert np.all(np.abs(np64(b) - e) <= rel * np.abs(e) + 2.0 ** -133)
        touched[b.storage_offset():b.storage_offset() + b.numel()] = True
    assert (dst[~touched] == 7.0).all()


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("power", [-133, -126, -100, -75, -64, -40, 60, 64, 90, 120])
def test_values_whose_squares_leave_fp32(kind, power):
    rng = np.random.default_rng(power + 200)
    t = torch.bfloat16 if kind == "bf16" else torch.float32
    a = torch.from_numpy(np.ldexp(rng.standard_normal(5000), power).astype(np.float32)).cuda().to(t)
    for g in ([a], [a, torch.zeros(3000, dtype=t, device="cuda"), a[:77]]):
        want = R.norm([np64(v) for v in g])
        assert want > 0
        got = float(mx.grad_norm(g))
        assert abs(got - want) <= NORM * want + 2.0 ** -150
        out = [torch.empty_like(v) for v in g]
        mx.clip_grads(g, 1e-3 * float(np.float32(want)) if power > -120 else 1.0, eps=0.0, out=out)
        c = R.factor(want, 1e-3 * float(np.float32(want)) if power > -120 else 1.0, 0.0)
        for v, o in zip(g, out):
            e = np64(v) * c
            # two products in fp32 where the factor is below 2^-100 (there is none here), one else; results below 2^-126 lose their last bits
            assert np.all(np.abs(np64(o) - e) <= (FACTOR + 2 * F32 + B16 * 1.01) * np.abs(e) + (2.0 ** -133 if kind == "bf16" else 2.0 ** -149))


def test_a_factor_below_the_normal_range():
    g = torch.full((4096,), 3e38, device="cuda")
    norm = R.norm([np64(g)])
    out = torch.empty_like(g)
    # (64 * 3e38: a norm that fp32 does not hold comes back as infinity, the factor follows the 64-bit one)
    assert float(mx.clip_grads([g], 1e-3, out=[out])) == float("inf")
    want = np64(g) * R.factor(norm, 1e-3)
    assert np.all(np.abs(np64(out) - want) <= (FACTOR + 2 * F32) * np.abs(want))
    g = torch.full((1 << 20,), 3e38, device="cuda")
    out = torch.empty_like(g)
    assert float(mx.clip_grads([g], 1.0, out=[out])) == float("inf")
    want = np64(g) * R.factor(R.norm([np64(g)]), 1.0)
    assert np.all(np.abs(np64(out) - want) <= (FACTOR + 2 * F32) * np.abs(want))


def test_zeros():
    for g in ([torch.zeros(1000, device="cuda")], [-torch.zeros(5, device="cuda"), torch.zeros(0, device="cuda", dtype=torch.bfloat16)]):
        assert float(mx.grad_norm(g)) == 0.0
        out = [torch.ones_like(t) for t in g]
        assert float(mx.clip_grads(g, 0.0, eps=1e-6, out=out)) == 0.0 and not any(o.any() for o in out)
        # 0 / 0: the factor is NaN
        mx.clip_grads(g, 0.0, eps=0.0, out=out)
        assert all(torch.isnan(o).all() for o in out)
    empty = [torch.zeros(0, device="cuda")]
    assert float(mx.grad_norm(empty)) == 0.0 and float(mx.clip_grads(empty, 1.0)) == 0.0
    norm = torch.full((), 9.0, device="cuda")
    assert float(mx.grad_norm([], out=norm)) == 0.0


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("at", [0, 8191, 40000])
def test_nan_and_infinity(kind, at):
    t = torch.bfloat16 if kind == "bf16" else torch.float32
    a, b = torch.randn(40001, device="cuda").to(t), torch.randn(1000, device="cuda").to(t)
    a[at] = float("inf")
    assert float(mx.grad_norm([b, a])) == float("inf")
    out = [torch.empty_like(v) for v in (a, b)]
    mx.clip_grads([a, b], 1.0, out=out)
    assert torch.isnan(out[0][at]) and int(torch.isnan(out[0]).sum()) == 1 and not out[1].any()
    a[at] = float("nan")
    b[3] = float("inf")
    assert np.isnan(float(mx.grad_norm([b, a])))
    mx.clip_grads([a, b], 1.0, out=out)
    assert torch.isnan(out[0]).all() and torch.isnan(out[1]).all()
    inplace = [a.clone(), b.clone()]
    mx.clip_grads(inplace, 1.0)
    assert torch.isnan(inplace[0]).all() and torch.isnan(inplace[1]).all()


def test_a_norm_that_is_known():
    g = [torch.randn(5000, device="cuda").bfloat16(), torch.randn(70, device="cuda")]
    before = [t.clone() for t in g]
    norm = torch.tensor(8.0, device="cuda")
    assert mx.clip_grads(g, 2.0, norm=norm, eps=0.0) is norm and float(norm) == 8.0
    assert all(torch.equal(a, b * 0.25) for a, b in zip(g, before))
    mx.clip_grads(g, 9.0, norm=norm)
    assert all(torch.equal(a, b * 0.25) for a, b in zip(g, before))
    many = [torch.randn(50, device="cuda") for _ in range(1500)]
    kept = [t.clone() for t in many]
    mx.clip_grads(many, 2.0, norm=norm, eps=0.0)
    assert all(torch.equal(a, b * 0.25) for a, b in zip(many, kept))


@pytest.mark.parametrize("n", [5000, 60_000_000])
@pytest.mark.parametrize("inplace", [True, False])
def test_a_norm_that_is_known_few_and_many_elements(n, inplace):
    """The same factor on both sides of the rule for many elements, with the cache's scratch and with a workspace."""
    g = [torch.randn(n, device="cuda").bfloat16(), torch.randn(n // 3 + 1, device="cuda")]
    norm = torch.tensor(3.0, device="cuda")
    c = R.factor(3.0, 1.0)
    ws = torch.empty(mx.grad_workspace_bytes(2), dtype=torch.uint8, device="cuda")
    for workspace in (None, ws):
        src = [t.clone() for t in g]
        out = None if inplace else [torch.full_like(t, 9.0) for t in g]
        mx.clip_grads(src, 1.0, norm=norm, out=out, workspace=workspace)
        for a, b in zip(src if inplace else out, g):
            want = b.double() * c
            rel = 2 * F32 * 1.001 + (B16 * 1.01 if b.dtype is torch.bfloat16 else 0.0)
            assert ((a.double() - want).abs() <= rel * want.abs() + 2.0 ** -133).all()
        assert float(norm) == 3.0


def test_a_tensor_twice():
    """Counted twice by the norm; as something to clip refused."""
    a = torch.randn(1000, device="cuda")
    assert abs(float(mx.grad_norm([a, a])) - np.sqrt(2) * float(a.double().norm())) < 1e-4
    with pytest.raises(mx.Mxfp8Error, match="overlaps"):
        mx.clip_grads([a, a], 1.0)
    with pytest.raises(mx.Mxfp8Error, match="overlaps"):
        mx.clip_grads([a[:600], a[599:]], 1.0)


def test_streams_graphs_and_workspaces():
    rng = np.random.default_rng(5)
    sets = [tensors(rng, [100000, 33, 70001], scale=s) for s in (1.0, 30.0)]
    want = []
    for g in sets:
        out = [torch.empty_like(t) for t in g]
        want.append((mx.clip_grads(g, 10.0, out=out), out))
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for g, s in zip(sets, streams):
            out = [torch.empty_like(t) for t in g]
            torch.cuda.synchronize()
            got.append((mx.clip_grads(g, 10.0, out=out, stream=s), out, mx.grad_norm(g, stream=s)))
    torch.cuda.synchronize()
    for (n, out, n2), (m, wout) in zip(got, want):
        assert float(n) == float(n2) == float(m) and all(torch.equal(a, b) for a, b in zip(out, wout))
    # two graphs with a workspace each, replayed in turn on changing inputs
    ws = [torch.empty(mx.grad_workspace_bytes(3), dtype=torch.uint8, device="cuda") for _ in sets]
    live = [[t.clone() for t in sets[0]] for _ in sets]
    outs = [[torch.empty_like(t) for t in sets[0]] for _ in sets]
    graphs, norms = [], []
    for g, o, w in zip(live, outs, ws):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            norms.append(mx.clip_grads(g, 10.0, out=o, workspace=w))
    for turn in range(2):
        for k in range(2):
            src = sets[(k + turn) % 2]
            for a, b in zip(live[k], src):
                a.copy_(b)
            graphs[k].replay()
        torch.cuda.synchronize()
        for k in range(2):
            m, wout = want[(k + turn) % 2]
            assert float(norms[k]) == float(m) and all(torch.equal(a, b) for a, b in zip(outs[k], wout))


def test_large_tensors():
    """More than 2^31 elements in a tensor, a few strong ones at its far end."""
    n = (1 << 31) + 12345
    a = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    a[-5:] = 3.0
    a[7] = 4.0
    want = np.sqrt(5 * 9 + 16)
    assert abs(float(mx.grad_norm([a])) - want) <= NORM * want
    mx.clip_grads([a], want / 2, eps=0.0)
    assert torch.equal(a[-5:], torch.full((5,), 1.5, dtype=torch.bfloat16, device="cuda")) and float(a[7]) == 2.0
    assert int(a.count_nonzero()) == 6
