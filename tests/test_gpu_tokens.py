"""Tokens sorted by expert and back on the GPU, against 64-bit implementations: plans bit for bit, rows bit for bit,
sums and gradients within what their roundings allow."""
import numpy as np
import pytest
import torch

import oracle
import moe_ragged_contraction_gb300 as mx
from moe_ragged_contraction_gb300 import _lib
import _step_ref as R

pytestmark = pytest.mark.gpu

# half a step of bf16, and of fp32, relative to the value
B16, F32 = torch.finfo(torch.bfloat16).eps / 2, torch.finfo(torch.float32).eps / 2
TINY = 2.0 ** -133  # half of bf16's smallest subnormal, where relative steps end


@pytest.fixture(scope="module", autouse=True)
def _lib_built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.build()
    yield
    assert mx.device_status(clear=True) == 0


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def np64(t):
    return t.double().cpu().numpy()


def bf16(rng, *shape):
    """Values of different strength by row, as bf16 on the GPU."""
    a = rng.standard_normal(shape) * np.exp(rng.standard_normal((*shape[:-1], 1)))
    return dev(a.astype(np.float32)).bfloat16()


def routing(kind, rng, T, k, experts):
    if kind == "spread":  # different experts a token, uneven
        score = rng.standard_normal((T, experts)) + rng.standard_normal(experts)
        ids = np.argsort(-score, axis=1)[:, :k]
        return ids if ids.shape[1] == k else rng.integers(0, experts, (T, k))
    if kind == "one":     # every pair to one expert, the same index again and again
        return np.full((T, k), experts // 2)
    if kind == "none":    # nothing here
        return rng.choice([-1, -7, experts, 2 ** 31 - 1], (T, k))
    if kind == "mixed":   # repeated experts, absent pairs, padding tokens at the end
        ids = rng.integers(-2, experts + 2, (T, k))
        ids[T - T // 5:] = -1
        return ids
    raise AssertionError(kind)


def make(rng, kind, T, k, experts, first, local, align, dtype=torch.int32, spare=0):
    ids = routing(kind, rng, T, k, experts)
    rows = mx.token_plan_rows(T, k, local, align) + spare * align
    plan = mx.token_plan(dev(ids).to(dtype), local, first_expert=first, align=align, rows=rows)
    return ids, rows, plan


SIZES = [  # kind, T, k, experts, first, local, align
    ("spread", 1, 1, 1, 0, 1, 1), ("spread", 1, 2, 4, 0, 4, 32), ("mixed", 3, 5, 4, 1, 2, 7), ("one", 33, 1, 9, 0, 9, 128),
    ("none", 40, 3, 8, 2, 4, 32), ("spread", 257, 8, 64, 16, 32, 32), ("mixed", 1000, 6, 64, 0, 64, 32), ("mixed", 130, 64, 100, 10, 80, 1),
    ("one", 5000, 8, 256, 120, 32, 32), ("spread", 4099, 4, 2048, 0, 2048, 32), ("mixed", 777, 33, 1600, 3, 1597, 256), ("spread", 20011, 8, 256, 96, 32, 1024),
]


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("kind,T,k,experts,first,local,align", SIZES)
def test_plan(kind, T, k, experts, first, local, align, dtype):
    rng = np.random.default_rng(T + k)
    ids, rows, plan = make(rng, kind, T, k, experts, first, local, align, dtype, spare=3)
    offs, slot, src, dropped = R.plan(ids, first, local, align, rows)
    assert dropped == 0
    for got, want in zip(plan, (offs, slot, src)):
        assert np.array_equal(got.cpu().numpy(), want)


def test_plan_of_wide_indices():
    """Indices beyond 32 bits are absent, not taken modulo 2^32."""
    ids = np.array([[0, 2 ** 32], [2 ** 40 + 1, 1], [-(2 ** 32), -(2 ** 63)], [2 ** 63 - 1, 1]])
    plan = mx.token_plan(dev(ids), 2, align=1, rows=8)
    offs, slot, src, _ = R.plan(ids, 0, 2, 1, 8)
    assert np.array_equal(plan.slot.cpu().numpy(), slot) and np.array_equal(plan.offs.cpu().numpy(), offs) and np.array_equal(plan.src.cpu().numpy(), src)


@pytest.mark.parametrize("T,k,local,align,rows", [(100, 4, 8, 32, 64), (100, 4, 8, 32, 0), (3000, 8, 40, 1, 10007), (50, 2, 4, 128, 256)])
def test_plan_with_too_few_rows(T, k, local, align, rows):
    rng = np.random.default_rng(rows)
    ids = rng.integers(0, local, (T, k))
    offs, slot, src, dropped = R.plan(ids, 0, local, align, rows)
    assert dropped > 0
    plan = mx.token_plan(dev(ids).int(), local, align=align, rows=rows)
    assert mx.device_status(clear=True) == _lib.DEV_TOKENS_ROWS
    for got, want in zip(plan, (offs, slot, src)):
        assert np.array_equal(got.cpu().numpy(), want)
    # dropped pairs are absent for every operator
    x = bf16(rng, T, 16)
    assert np.array_equal(np64(mx.token_dispatch(x, plan)), R.dispatch(np64(x), src, k))


@pytest.mark.parametrize("T,k,experts,first,local,align", [(300000, 4, 64, 0, 64, 32), (150001, 8, 2100, 40, 2048, 1), (530000, 2, 8, 1, 6, 128), (1100000, 1, 1, 0, 1, 32)])
def test_plan_of_long_runs(T, k, experts, first, local, align):
    """More pairs than the kernel keeps ranks of at a time."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)
    ids = torch.randint(-1 if experts > 1 else 0, experts, (T, k), generator=gen, device="cuda")
    plan = mx.token_plan(ids, local, first_expert=first, align=align)
    e = ids.view(-1) - first
    here = (e >= 0) & (e < local)
    count = torch.bincount(e[here], minlength=local)
    padded = (count + align - 1) // align * align
    offs = torch.cumsum(padded, 0)
    order = torch.nonzero(here).squeeze(-1)[torch.sort(e[here], stable=True).indices]
    starts = torch.repeat_interleave(offs - padded, count)
    row = starts + torch.arange(len(order), device="cuda") - torch.repeat_interleave(torch.cumsum(count, 0) - count, count)
    slot = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
    src = torch.full((plan.src.numel(),), -1, dtype=torch.int32, device="cuda")
    slot[order], src[row] = row.int(), order.int()
    assert torch.equal(plan.offs.long(), offs) and torch.equal(plan.slot.view(-1), slot) and torch.equal(plan.src, src)
    # with too few rows
    rows = int(offs[-1]) // 2 // align * align
    short = mx.token_plan(ids, local, first_expert=first, align=align, rows=rows)
    assert mx.device_status(clear=True) == _lib.DEV_TOKENS_ROWS
    assert torch.equal(short.slot.view(-1), torch.where(slot < rows, slot, -1)) and torch.equal(short.src, src[:rows])


@pytest.mark.parametrize("T", [0, 1, 31, 5000])
def test_plan_fills_what_it_is_given(T):
    """Every element of the outputs is written, with many rows to spare; no token at all among the sizes."""
    ids = torch.zeros((T, 2), dtype=torch.int32, device="cuda")
    rows = mx.token_plan_rows(T, 2, 3, 32) + 100000 // 32 * 32
    out = mx.TokenPlan(*(torch.full(s, 12345, dtype=torch.int32, device="cuda") for s in ((3,), (T, 2), (rows,))))
    assert mx.token_plan(ids, 3, out=out) == out
    offs, slot, src, _ = R.plan(ids.cpu().numpy(), 0, 3, 32, rows)
    for got, want in zip(out, (offs, slot, src)):
        assert np.array_equal(got.cpu().numpy(), want)


ROWS = [  # kind, T, k, experts, first, local, align, H
    ("spread", 1, 2, 4, 0, 4, 32, 256), ("spread", 1, 1, 1, 0, 1, 1, 8), ("mixed", 3, 5, 4, 1, 2, 7, 40), ("none", 40, 3, 8, 2, 4, 32, 96),
    ("one", 33, 1, 9, 0, 9, 128, 1032), ("mixed", 130, 64, 100, 10, 80, 1, 72), ("spread", 257, 8, 64, 16, 32, 32, 7168), ("mixed", 1000, 6, 64, 0, 64, 32, 2048),
    ("mixed", 61, 33, 40, 3, 37, 16, 512), ("spread", 5, 4, 8, 0, 8, 32, 32768), ("spread", 2000, 3, 21, 4, 13, 32, 1096),
]


@pytest.mark.parametrize("kind,T,k,experts,first,local,align,H", ROWS)
def test_dispatch(kind, T, k, experts, first, local, align, H):
    rng = np.random.default_rng(H + T)
    ids, rows, plan = make(rng, kind, T, k, experts, first, local, align, spare=2)
    x = bf16(rng, T, H)
    x.view(-1)[0] = float("nan")
    x.view(-1)[-1] = float("-inf")
    out = torch.full((rows, H), 7.0, dtype=torch.bfloat16, device="cuda")
    assert mx.token_dispatch(x, plan, out=out) is out
    src = plan.src.cpu().numpy()
    assert np.array_equal(out.view(torch.int16).cpu().numpy(), R.dispatch(x.view(torch.int16).cpu().numpy(), src, k))


@pytest.mark.parametrize("kind,T,k,experts,first,local,align,H", [(*r[:7], max(32, r[7] // 32 * 32)) for r in ROWS])
def test_dispatch_mxfp8(kind, T, k, experts, first, local, align, H):
    rng = np.random.default_rng(H + T)
    ids, rows, plan = make(rng, kind, T, k, experts, first, local, align, spare=2)
    a = rng.standard_normal((T, H)) * np.exp2(rng.integers(-20, 20, (T, H)))
    a[rng.random((T, H)) < 0.2] = 0.0
    a[0, :32] = 0.0                      # a block of zeros (of either sign)
    a[0, 3] = -0.0
    if H >= 64:
        a[-1, 32:64] *= 2.0 ** -126      # subnormal blocks
    x = dev(a.astype(np.float32)).bfloat16()
    if T > 2:
        x[1, 5], x[2, -1] = float("nan"), float("inf")
        x[2, 0] = 3.3895e38
    q, s = mx.token_dispatch_mxfp8(x, plan)
    want_q, want_s = oracle.quantize_tokenwise(np.ascontiguousarray(x.float().cpu().numpy()))
    src = plan.src.cpu().numpy()
    assert np.array_equal(q.cpu().numpy(), R.dispatch(want_q, src, k))
    assert np.array_equal(s.cpu().numpy(), R.dispatch(want_s, src, k))


def with_rubbish(y, w, plan):
    """NaN where nothing may be read: padding rows, weights of absent pairs."""
    y[plan.src < 0] = float("nan")
    if w is not None:
        w[plan.slot < 0] = float("nan")


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("kind,T,k,experts,first,local,align,H", ROWS)
def test_combine(kind, T, k, experts, first, local, align, H, weighted):
    rng = np.random.default_rng(H + T + 1)
    ids, rows, plan = make(rng, kind, T, k, experts, first, local, align, spare=2)
    y, w = bf16(rng, rows, H), dev(rng.random((T, k)).astype(np.float32) - 0.2)
    with_rubbish(y, w, plan)
    out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    if weighted:
        mx.token_combine(y, w, plan, out=out)
    else:
        mx.token_dispatch_grad(y, plan, out=out)
    want, mag = R.combine(np64(y), np64(w) if weighted else None, plan.slot.cpu().numpy())
    # k products and sums in fp32, then one rounding to bf16 (of a value that far off)
    sums = 2 * k * F32 * mag
    assert np.all(np.abs(np64(out) - want) <= sums + B16 * (np.abs(want) + sums) + TINY)
    empty = (plan.slot.cpu().numpy() < 0).all(1)
    assert not out.view(torch.int16).cpu().numpy()[empty].any()


@pytest.mark.parametrize("kind,T,k,experts,first,local,align,H", ROWS)
def test_combine_grad(kind, T, k, experts, first, local, align, H):
    rng = np.random.default_rng(H + T + 2)
    ids, rows, plan = make(rng, kind, T, k, experts, first, local, align, spare=2)
    y, w, dout = bf16(rng, rows, H), dev(rng.random((T, k)).astype(np.float32) - 0.2), bf16(rng, T, H)
    with_rubbish(y, w, plan)
    dy = torch.full((rows, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    dw = torch.full((T, k), float("nan"), device="cuda")
    mx.token_combine_grad(dout, y, w, plan, dy=dy, dweights=dw)
    slot, src = plan.slot.cpu().numpy(), plan.src.cpu().numpy()
    want, want_w, mag = R.combine_grad(np64(dout), np64(y), np64(w), slot, rows)
    assert np.all(np.abs(np64(dy) - want) <= (B16 + 2 * F32) * np.abs(want) + TINY)
    assert not dy.view(torch.int16).cpu().numpy()[src < 0].any()
    # a lane's chain of 8 columns in 256, the lanes' sums in five steps more
    steps = 8 * -(-H // 256) + 6
    assert np.all(np.abs(np64(dw) - want_w) <= steps * F32 * mag)
    assert not dw.view(torch.int32).cpu().numpy()[slot < 0].any()
    # over y itself
    again, dw2 = mx.token_combine_grad(dout, y, w, plan, dy=y)
    assert again is y and torch.equal(y.view(torch.int16), dy.view(torch.int16)) and torch.equal(dw2, dw)


def test_empty_buffers():
    """No tokens, no rows, neither."""
    for T, rows in ((0, 64), (0, 0), (3, 0)):
        plan = mx.token_plan(torch.full((T, 2), -1, dtype=torch.int32, device="cuda"), 2, rows=rows)
        x = torch.ones((T, 64), dtype=torch.bfloat16, device="cuda")
        assert not mx.token_dispatch(x, plan).any() and mx.token_dispatch(x, plan).shape == (rows, 64)
        q, s = mx.token_dispatch_mxfp8(x, plan)
        assert q.shape == (rows, 64) and not q.any() and not s.any()
        y, w = torch.ones((rows, 64), dtype=torch.bfloat16, device="cuda"), torch.ones((T, 2), device="cuda")
        assert not mx.token_dispatch_grad(y, plan).any() and not mx.token_combine(y, w, plan).any()
        dy, dw = mx.token_combine_grad(x, y, w, plan)
        assert dy.shape == (rows, 64) and not dy.any() and not dw.any()


def test_plans_that_are_no_plans():
    """Entries out of range count as absent, wherever they point."""
    T, k, rows, H = 5, 3, 40, 64
    rng = np.random.default_rng(4)
    slot = np.array([[0, 40, 1], [-2, 2, 2 ** 31 - 1], [-(2 ** 31), 3, 41], [4, 5, 6], [7, 1000, -1]], np.int32)
    src = np.full(rows, -1, np.int32)
    src[:8] = [0, 2, 4, 7, 9, 10, 11, 12]
    src[8:12] = [15, 2 ** 31 - 1, -5, -(2 ** 31)]
    ok_slot, ok_src = np.where((slot >= 0) & (slot < rows), slot, -1), np.where((src >= 0) & (src < T * k), src, -1)
    bad, good = (mx.TokenPlan(dev(np.zeros(1, np.int32)), dev(a), dev(b)) for a, b in ((slot, src), (ok_slot, ok_src)))
    x, y, w = bf16(rng, T, H), bf16(rng, rows, H), dev(rng.random((T, k)).astype(np.float32))
    for f in (lambda p: mx.token_dispatch(x, p), lambda p: mx.token_dispatch_mxfp8(x, p), lambda p: mx.token_dispatch_grad(y, p),
              lambda p: mx.token_combine(y, w, p), lambda p: mx.token_combine_grad(x, y, w, p)):
        want = f(good)
        assert mx.device_status(clear=True) == 0
        got = f(bad)
        assert mx.device_status(clear=True) == _lib.DEV_TOKENS_RANGE
        for a, b in zip(got if isinstance(got, tuple) else (got,), want if isinstance(want, tuple) else (want,)):
            assert torch.equal(a, b)


def test_nan_and_infinity_in_rows_and_weights():
    """They reach the tokens that own them and no others."""
    T, k, H = 40, 2, 96
    rng = np.random.default_rng(8)
    ids = np.stack([np.arange(T) % 5, 5 + np.arange(T) % 3], 1)
    plan = mx.token_plan(dev(ids).int(), 8)
    y, w = bf16(rng, plan.src.numel(), H), dev(rng.random((T, k)).astype(np.float32) + 0.1)
    slot = plan.slot.cpu().numpy()
    y[slot[3, 0], 7] = float("nan")
    y[slot[4, 1], 9] = float("inf")
    w[5, 0] = float("nan")
    out = np64(mx.token_combine(y, w, plan))
    odd = ~np.isfinite(out)
    want = np.zeros_like(odd)
    want[3, 7] = want[4, 9] = True
    want[5] = True
    assert np.array_equal(odd, want) and np.isposinf(out[4, 9])
    dy, dw = mx.token_combine_grad(torch.ones((T, H), dtype=torch.bfloat16, device="cuda"), y, w, plan)
    dy, dw = np64(dy), np64(dw)
    assert np.isnan(dy[slot[5, 0]]).all() and np.isfinite(np.delete(dy, slot[5, 0], 0)).all()
    assert np.isnan(dw[3, 0]) and np.isposinf(dw[4, 1]) and np.isfinite(dw).sum() == T * k - 2


@pytest.mark.parametrize("shift", [1, 2, 3])
def test_views_of_larger_buffers(shift):
    """Inputs and outputs that start 16 bytes apart inside a buffer; what lies around an output stays as it was."""
    T, k, H = 37, 3, 40
    rng = np.random.default_rng(shift)
    ids = rng.integers(-1, 6, (T, k))
    plan = mx.token_plan(dev(ids).int(), 5, first_expert=1, align=4)
    rows = plan.src.numel()

    def view(n, m):
        whole = torch.full((n * m + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
        return whole, whole[8 * shift:8 * shift + n * m].view(n, m)

    x0, x = view(T, H)
    x.copy_(bf16(rng, T, H))
    o0, o = view(rows, H)
    mx.token_dispatch(x, plan, out=o)
    assert torch.equal(o, mx.token_dispatch(x.clone(), plan))
    c0, c = view(T, H)
    mx.token_dispatch_grad(o, plan, out=c)
    assert torch.equal(c, mx.token_dispatch_grad(o.clone(), plan))
    d0, d = view(rows, H)
    w = torch.rand((T, k), device="cuda")
    mx.token_combine_grad(x, o, w, plan, dy=d)
    for whole, n in ((o0, rows * H), (c0, T * H), (d0, rows * H)):
        assert (whole[:8 * shift] == 3.0).all() and (whole[8 * shift + n:] == 3.0).all()


@pytest.mark.parametrize("shift", [1, 2, 3, 4])
@pytest.mark.parametrize("H", [256, 2176])
def test_scales_at_any_address(shift, H):
    """Scale planes need no alignment: by words and by bytes, nothing written around them."""
    rng = np.random.default_rng(H)
    T, k = 50, 3
    plan = mx.token_plan(dev(rng.integers(-1, 4, (T, k))).int(), 4)
    rows = plan.src.numel()
    x = bf16(rng, T, H)
    q, s = mx.token_dispatch_mxfp8(x, plan)
    whole = torch.full((rows * H // 32 + 8,), 77, dtype=torch.uint8, device="cuda")
    view = whole[shift:shift + rows * H // 32].view(rows, H // 32)
    q2, _ = mx.token_dispatch_mxfp8(x, plan, s=view)
    assert torch.equal(q, q2) and torch.equal(s, view)
    assert (whole[:shift] == 77).all() and (whole[shift + rows * H // 32:] == 77).all()


def test_results_are_the_same_bits_every_time():
    rng = np.random.default_rng(11)
    ids = dev(routing("spread", rng, 3000, 8, 64)).int()
    x = bf16(rng, 3000, 2048)
    w = torch.rand((3000, 8), device="cuda")
    first = None
    for _ in range(3):
        plan = mx.token_plan(ids, 64)
        xs = mx.token_dispatch(x, plan)
        out = mx.token_combine(xs, w, plan)
        dy, dw = mx.token_combine_grad(out, xs, w, plan)
        dx = mx.token_dispatch_grad(dy, plan)
        got = (*plan, xs, out, dy, dw, dx)
        if first is not None:
            assert all(torch.equal(a, b) for a, b in zip(first, got))
        first = got


def test_other_streams_and_graphs():
    """On a stream of its own beside another call, and captured, replayed on other inputs in the same buffers."""
    rng = np.random.default_rng(12)
    T, k, H = 700, 4, 1024
    ids = [dev(rng.integers(0, 16, (T, k))).int() for _ in range(3)]
    x, w = bf16(rng, T, H), torch.rand((T, k), device="cuda")

    def chain(ids, x, w, stream=None):
        plan = mx.token_plan(ids, 16, stream=stream)
        xs = mx.token_dispatch(x, plan, stream=stream)
        q, s = mx.token_dispatch_mxfp8(x, plan, stream=stream)
        out = mx.token_combine(xs, w, plan, stream=stream)
        dy, dw = mx.token_combine_grad(out, xs, w, plan, stream=stream)
        return (*plan, xs, q, s, out, dy, dw, mx.token_dispatch_grad(dy, plan, stream=stream))

    want = [chain(i, x, w) for i in ids]
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        got = chain(ids[0], x, w, a), chain(ids[1], x, w, b)
    torch.cuda.synchronize()
    for g, e in zip(got, want):
        assert all(torch.equal(u, v) for u, v in zip(g, e))
    live, lx, lw = ids[0].clone(), x.clone(), w.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(live, lx, lw)
    for i in (2, 0, 1):
        live.copy_(ids[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(out, want[i]))


def test_offsets_beyond_32_bits():
    """Sorted buffers of more than 2^31 elements and 2^32 bytes: rows at their far end."""
    H, k, T = 32768, 2, 64
    rows = 70016  # times H: 2.29e9 elements, 4.6 GB
    experts = 2000
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    filler = torch.zeros((rows // k - T - 32, k), dtype=torch.int32, device="cuda")  # expert 0 takes all but the last rows
    ids[:, 0] = torch.arange(T, dtype=torch.int32, device="cuda") % 3
    ids = torch.cat((filler, ids + (ids >= 0) * (experts - 3)))
    plan = mx.token_plan(ids, experts, align=1, rows=rows)
    far = plan.slot[-T:, 0].long()
    assert int(far.min()) * H > 2 ** 31
    x = torch.zeros((ids.shape[0], H), dtype=torch.bfloat16, device="cuda")
    x[-T:] = torch.randn((T, H), device="cuda").bfloat16()
    xs = torch.full((rows, H), 9.0, dtype=torch.bfloat16, device="cuda")
    mx.token_dispatch(x, plan, out=xs)
    assert torch.equal(xs[far], x[-T:]) and not xs[int(far.max()) + 1:].any()
    back = mx.token_dispatch_grad(xs, plan)
    assert torch.equal(back[-T:], x[-T:])
    w = torch.full((ids.shape[0], k), 0.5, device="cuda")
    out = mx.token_combine(xs, w, plan)
    assert torch.equal(out[-T:], x[-T:] * 0.5)
    q, s = mx.token_dispatch_mxfp8(x, plan)
    qx, sx = mx.quantize_tokenwise(x[-T:].float())
    assert torch.equal(q[far], qx) and torch.equal(s[far], sx)
    dy, dw = mx.token_combine_grad(x, xs, w, plan, dy=xs)
    assert torch.equal(dy[far], x[-T:] * 0.5)
    want = x[-T:].double().square().sum(-1)
    assert ((dw[-T:, 0].double() - want).abs() <= (8 * H // 256 + 6) * F32 * want).all() and not dw[-T:, 1].any()
