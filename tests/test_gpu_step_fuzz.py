"""Random routings, sizes and lists of gradients through the operators of a training step, against 64 bits (vectorised)."""
import random

import numpy as np
import pytest
import torch

import moe_ragged_contraction_gb300 as mx
import _step_ref as R

pytestmark = pytest.mark.gpu

B16, F32 = torch.finfo(torch.bfloat16).eps / 2, torch.finfo(torch.float32).eps / 2
TINY = 2.0 ** -133


@pytest.fixture(scope="module", autouse=True)
def _lib_built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.build()
    yield
    assert mx.device_status(clear=True) == 0


def log(r, lo, hi):
    return round(np.exp(r.uniform(np.log(lo), np.log(hi))))


@pytest.mark.parametrize("seed", range(40))
def test_tokens(seed):
    r = random.Random(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    T, k = log(r, 1, 60000), log(r, 1, 64)
    T = max(1, min(T, 400000 // k))
    H = min(8 * log(r, 1, 1024), max(8, 30_000_000 // (T * k) // 8 * 8))
    local = log(r, 1, 2048)
    experts = min(4 * 2048, round(local * r.choice((1, 1, 2, 9))))
    first, align = r.randint(0, experts - local), r.choice((1, 32, 32, r.randint(2, 1024)))
    if local * align * H > 200_000_000:
        align = 1
    ids = torch.randint(-1 if r.random() < 0.5 else 0, experts, (T, k), generator=gen, device="cuda")
    if r.random() < 0.3:
        ids = ids // r.randint(2, 50)  # few experts, many pairs each
    if r.random() < 0.5:
        ids = ids.int()
    rows = mx.token_plan_rows(T, k, local, align)
    plan = mx.token_plan(ids, local, first_expert=first, align=align)
    # the plan, by sorting
    e = ids.cpu().numpy().astype(np.int64).reshape(-1) - first
    here = (e >= 0) & (e < local)
    count = np.bincount(e[here], minlength=local)
    padded = -(-count // align) * align
    offs = np.cumsum(padded)
    order = np.flatnonzero(here)[np.argsort(e[here], kind="stable")]
    row = np.repeat(offs - padded, count) + np.arange(len(order)) - np.repeat(np.cumsum(count) - count, count)
    slot, src = np.full(T * k, -1, np.int32), np.full(rows, -1, np.int32)
    slot[order], src[row] = row, order
    assert np.array_equal(plan.offs.cpu().numpy(), offs)
    assert np.array_equal(plan.slot.cpu().numpy().reshape(-1), slot) and np.array_equal(plan.src.cpu().numpy(), src)

    bf = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    x, y, dout, w = bf(T, H), bf(rows, H), bf(T, H), torch.rand((T, k), generator=gen, device="cuda") - 0.3
    y[plan.src < 0] = float("nan")
    w[plan.slot < 0] = float("nan")
    dsrc = plan.src.long()
    want = torch.where((dsrc >= 0)[:, None], x[dsrc.clamp(min=0) // k], torch.zeros((), dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(mx.token_dispatch(x, plan), want)
    if H % 32 == 0:
        q, s = mx.token_dispatch_mxfp8(x, plan)
        wq, ws = mx.quantize_tokenwise(want.float()) if rows else (q, s)
        assert torch.equal(q, wq) and torch.equal(s, ws)
    pair = torch.from_numpy(order).cuda()
    at, token, y64 = torch.from_numpy(row).cuda(), pair // k, y.double()
    for weighted in (False, True):
        terms = y64[at] * (w.double().reshape(-1)[pair, None] if weighted else 1.0)
        ref = torch.zeros((T, H), dtype=torch.float64, device="cuda").index_add_(0, token, terms)
        mag = torch.zeros((T, H), dtype=torch.float64, device="cuda").index_add_(0, token, terms.abs())
        out = mx.token_combine(y, w, plan) if weighted else mx.token_dispatch_grad(y, plan)
        sums = 2 * k * F32 * mag
        assert ((out.double() - ref).abs() <= sums + B16 * (ref.abs() + sums) + TINY).all()
    dy, dw = mx.token_combine_grad(dout, y, w, plan)
    ref = torch.zeros((rows, H), dtype=torch.float64, device="cuda")
    ref[at] = w.double().reshape(-1)[pair, None] * dout.double()[token]
    assert ((dy.double() - ref).abs() <= (B16 + 2 * F32) * ref.abs() + TINY).all()
    prod = y64[at] * dout.double()[token]
    rdw, mag = torch.zeros(T * k, dtype=torch.float64, device="cuda"), torch.zeros(T * k, dtype=torch.float64, device="cuda")
    rdw[pair], mag[pair] = prod.sum(-1), prod.abs().sum(-1)
    assert ((dw.double().reshape(-1) - rdw).abs() <= (8 * -(-H // 256) + 6) * F32 * mag).all()


@pytest.mark.parametrize("seed", range(25))
def test_gradients(seed):
    r = random.Random(1000 + seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    n, total = log(r, 1, 2500), log(r, 1, 3_000_000)
    flat = {t: torch.full((2 * total + 4 * n + 64,), 7.0, dtype=t, device="cuda") for t in (torch.bfloat16, torch.float32)}
    at = {t: r.randint(0, 5) for t in flat}
    grads = []
    for _ in range(n):
        t = r.choice(list(flat))
        size = min(log(r, 1, max(2, 3 * total // n)) - 1, total)
        if at[t] + size > flat[t].numel():
            break
        v = flat[t][at[t]:at[t] + size]
        v.copy_(torch.randn(size, generator=gen, device="cuda") * 2.0 ** r.randint(-20, 10))
        at[t] += size + r.randint(0, 3)
        grads.append(v)
    before = {t: f.clone() for t, f in flat.items()}
    want = R.norm([g.double().cpu().numpy() for g in grads])
    norm = mx.grad_norm(grads)
    assert abs(float(norm) - want) <= 10.1 * F32 * want
    limit = want * r.choice((0.01, 0.7, 1.5)) + 1e-30
    c = R.factor(want, limit)
    assert float(mx.clip_grads(grads, limit)) == float(norm)
    touched = {t: torch.zeros_like(f, dtype=torch.bool) for t, f in flat.items()}
    for g in grads:
        touched[g.dtype][g.storage_offset():g.storage_offset() + g.numel()] = True
    for t, f in flat.items():
        assert torch.equal(f[~touched[t]], before[t][~touched[t]])
        ref = before[t][touched[t]].double() * c
        rel = 0.0 if c == 1.0 else 11.1 * F32 + (1.01 * B16 if t is torch.bfloat16 else 0.0)
        assert ((f[touched[t]].double() - ref).abs() <= rel * ref.abs() + TINY).all()


@pytest.mark.parametrize("T,k,local,experts", [(30, 4, 8, 8), (900, 8, 32, 32), (9000, 8, 8, 64), (20000, 4, 16, 16)])
def test_plans_with_entries_out_of_range(T, k, local, experts):
    """Every way in which the kernels share their work: an entry out of range counts as absent, and is reported."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)
    H = 96
    ids = torch.rand((T, experts), generator=gen, device="cuda").topk(k).indices
    rows = min(mx.token_plan_rows(T, k, local, 32), round(1.2 * T * k * local / experts / 32 + local + 8) * 32)
    good = mx.token_plan(ids, local, rows=rows)
    wild = lambda n: torch.randint(-2 ** 31, 2 ** 31 - 1, (n,), generator=gen, device="cuda", dtype=torch.int64).int()  # noqa: E731
    # the pairs of some rows lose both of their entries; the bad plan has wild ones in their places
    slot, src = good.slot.clone().view(-1), good.src.clone()
    lost = torch.nonzero(torch.rand(rows, generator=gen, device="cuda") < 0.2).squeeze(-1)
    pairs = src[lost].long()
    lost, pairs = lost[pairs >= 0], pairs[pairs >= 0]
    slot[pairs], src[lost] = -1, -1
    clean = mx.TokenPlan(good.offs, slot.view(T, k), src)
    bad_slot, bad_src = slot.clone(), src.clone()
    v = wild(len(lost))
    bad_slot[pairs] = torch.where((v < -1) | (v >= rows), v, rows + 5)
    v = wild(len(lost))
    bad_src[lost] = torch.where((v < -1) | (v >= T * k), v, -7)
    bad = mx.TokenPlan(good.offs, bad_slot.view(T, k), bad_src)
    bf = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    x, y, dout, w = bf(T, H), bf(rows, H), bf(T, H), torch.rand((T, k), generator=gen, device="cuda")
    assert mx.device_status(clear=True) == 0
    for f in (lambda p: [mx.token_dispatch(x, p)], lambda p: mx.token_dispatch_mxfp8(x, p), lambda p: [mx.token_dispatch_grad(y, p)],
              lambda p: [mx.token_combine(y, w, p)], lambda p: mx.token_combine_grad(dout, y, w, p)):
        want = f(clean)
        assert mx.device_status(clear=True) == 0
        got = f(bad)
        assert mx.device_status(clear=True) == 32
        assert all(torch.equal(a, b) for a, b in zip(got, want))
