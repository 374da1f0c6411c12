"""The ways that the token operators take for many tokens and wide rows: units of several trips, sums of one, three, six and
eight rows at a time, the gradient with lists of the pairs that are here. Against 64 bits, at sizes where the ways' last
trips, units and lists are parts."""
import pytest
import torch

import moe_ragged_contraction_gb300 as mx
from moe_ragged_contraction_gb300 import _lib

pytestmark = pytest.mark.gpu

B16, F32 = torch.finfo(torch.bfloat16).eps / 2, torch.finfo(torch.float32).eps / 2
TINY = 2.0 ** -133  # half of bf16's smallest subnormal, where relative steps end


@pytest.fixture(scope="module", autouse=True)
def _lib_built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.build()
    yield
    assert mx.device_status(clear=True) == 0


def routed(T, k, experts, local, seed, absent=0.0, rows=None, align=32):
    """Different experts of a token, some tokens without any (padding); a plan of experts 1 .. local."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    ids = torch.rand((T, experts), generator=gen, device="cuda").topk(k).indices if experts >= k else torch.randint(0, experts, (T, k), generator=gen, device="cuda")
    ids[torch.rand(T, generator=gen, device="cuda") < absent] = -1
    here = int(((ids >= 1) & (ids <= local)).sum())
    if rows is None:
        rows = (here + local * align) // align * align  # enough, and some rows behind the last group
    plan = mx.token_plan(ids, local, first_expert=1, align=align, rows=rows)
    return gen, plan


def rand(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").bfloat16()


def pairs_of(plan):
    """(pair, row) of what is here."""
    slot = plan.slot.view(-1).long()
    pair = torch.nonzero(slot >= 0).squeeze(-1)
    return pair, slot[pair]


def check_sums(gen, plan, T, k, H):
    """The sum with and without weights, NaN where nothing may be read."""
    pair, row = pairs_of(plan)
    y, w = rand(gen, plan.src.numel(), H), torch.rand((T, k), generator=gen, device="cuda") - 0.3
    y[plan.src < 0] = float("nan")
    w[plan.slot < 0] = float("nan")
    for weighted in (True, False):
        out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
        mx.token_combine(y, w, plan, out=out) if weighted else mx.token_dispatch_grad(y, plan, out=out)
        terms = y[row].double()
        if weighted:
            terms *= w.reshape(-1)[pair, None].double()
        want = torch.zeros((T, H), dtype=torch.float64, device="cuda").index_add_(0, pair // k, terms)
        sums = torch.zeros((T, H), dtype=torch.float64, device="cuda").index_add_(0, pair // k, terms.abs_())
        del terms
        sums *= 2 * k * F32  # k products and k sums in fp32, then one rounding to bf16 of a value that far off
        assert ((out.double() - want).abs_() <= sums + B16 * (want.abs() + sums) + TINY).all()
        assert not out.view(torch.int16)[(plan.slot < 0).all(1)].any()


# T, k, experts, local, H
SUMS = [
    (20011, 3, 5, 5, 520),      # units of 512 columns, the last of 8; three rows at a time, two vectors of each
    (41003, 3, 5, 5, 1032),     # whole tokens: three trips, the last of 8 columns
    (41003, 3, 9, 4, 776),      # the same with one row, two or none of many tokens
    (20011, 6, 8, 8, 1096),     # units of 512 columns: two trips of six rows, the last unit 72 columns
    (20011, 6, 24, 18, 2048),   # four to six rows
    (41003, 5, 6, 6, 1288),     # whole tokens: six trips of five rows
    (20011, 9, 12, 12, 776),    # eight rows and one more
    (20011, 8, 9, 9, 520),      # seven or eight
    (20011, 40, 80, 20, 264),   # choices beyond the 32nd
    (20011, 1, 3, 2, 2568),     # one row or none: whole tokens in two trips of 2048 columns
    (20011, 2, 9, 2, 4104),     # one row mostly, some two: whole tokens (20000 units are enough)
]


@pytest.mark.parametrize("T,k,experts,local,H", SUMS)
def test_sums(T, k, experts, local, H):
    gen, plan = routed(T, k, experts, min(local, experts), H, absent=0.05)
    check_sums(gen, plan, T, k, H)


@pytest.mark.parametrize("T,k,experts,local,H", [(41003, 3, 5, 5, 1032), (20011, 2, 9, 4, 2600), (20011, 1, 3, 3, 4104), (20011, 40, 80, 20, 264), (5003, 4, 8, 5, 2080), (5003, 3, 8, 8, 4128), (2500, 2, 4, 3, 8224)])
def test_rows(T, k, experts, local, H):
    """Rows in sorted order of several trips a unit, and to MXFP8 (units of 4096 and 8192 columns: trips of 2048)."""
    gen, plan = routed(T, k, experts, local, H + 1, absent=0.05)
    x = rand(gen, T, H)
    x.view(-1)[-1] = float("-inf")
    out = torch.full((plan.src.numel(), H), 7.0, dtype=torch.bfloat16, device="cuda")
    mx.token_dispatch(x, plan, out=out)
    src = plan.src.long()
    want = torch.where((src >= 0)[:, None], x[src.clamp(min=0) // k].view(torch.int16), torch.zeros((), dtype=torch.int16, device="cuda"))
    assert torch.equal(out.view(torch.int16), want)
    if H % 32:
        return
    q, s = mx.token_dispatch_mxfp8(x, plan)
    wq, ws = mx.quantize_tokenwise(want.view(torch.bfloat16).float())
    assert torch.equal(q, wq) and torch.equal(s, ws)


# The gradient with lists: more than 2048 columns, rows for less than half of the pairs, more than 64 x 4 pairs an SM.
LISTS = [
    (9001, 8, 64, 8, 2056),      # the last list of 8 pairs; two trips of a row, the second of 8 columns
    (9001, 8, 64, 8, 4104),      # two whole trips and 8 columns
    (40009, 1, 16, 3, 2312),     # one choice
    (5003, 33, 99, 20, 2064),    # choices beyond the 32nd; lists that end inside a token
    (20011, 2, 40, 1, 2176),     # lists with a pair or none
]


def check_gradient(plan, dout, y, w, dy, dw, k, H):
    pair, row = pairs_of(plan)
    want = torch.zeros(dy.shape, dtype=torch.float64, device="cuda")
    want[row] = w.reshape(-1)[pair, None].double() * dout[pair // k].double()
    assert ((dy.double() - want).abs_() <= (B16 + 2 * F32) * want.abs_() + TINY).all()
    assert not dy.view(torch.int16)[plan.src < 0].any()
    del want
    terms = y[row].double() * dout[pair // k].double()
    wanted, mag = torch.zeros(w.numel(), dtype=torch.float64, device="cuda"), torch.zeros(w.numel(), dtype=torch.float64, device="cuda")
    wanted[pair], mag[pair] = terms.sum(-1), terms.abs_().sum(-1)
    # a lane's chain of 8 columns in 256, the lanes' sums in five steps more
    assert ((dw.double().view(-1) - wanted).abs() <= (8 * -(-H // 256) + 6) * F32 * mag).all()
    assert not dw.view(torch.int32)[plan.slot < 0].any()


@pytest.mark.parametrize("T,k,experts,local,H", LISTS)
def test_gradient_with_lists(T, k, experts, local, H):
    gen, plan = routed(T, k, experts, local, H + 2, absent=0.05)
    rows = plan.src.numel()
    assert 2 * rows < T * k and T * k > 64 * 4 * torch.cuda.get_device_properties(0).multi_processor_count and H > 2048
    dout, y, w = rand(gen, T, H), rand(gen, rows, H), torch.rand((T, k), generator=gen, device="cuda") - 0.3
    y[plan.src < 0] = float("nan")
    w[plan.slot < 0] = float("nan")
    dy = torch.full((rows, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    dw = torch.full((T, k), float("nan"), device="cuda")
    mx.token_combine_grad(dout, y, w, plan, dy=dy, dweights=dw)
    check_gradient(plan, dout, y, w, dy, dw, k, H)
    # once more, and over y itself: the same bits
    again, dw2 = mx.token_combine_grad(dout, y, w, plan)
    assert torch.equal(again, dy) and torch.equal(dw2, dw)
    over, dw3 = mx.token_combine_grad(dout, y, w, plan, dy=y)
    assert over is y and torch.equal(y, dy) and torch.equal(dw3, dw)


def test_gradient_with_lists_of_pairs_that_were_dropped():
    """Too few rows: the dropped pairs are absent."""
    T, k, H = 9001, 8, 2056
    gen, plan = routed(T, k, 64, 8, 3, rows=6400)
    assert mx.device_status(clear=True) == _lib.DEV_TOKENS_ROWS
    dout, y, w = rand(gen, T, H), rand(gen, 6400, H), torch.rand((T, k), generator=gen, device="cuda")
    dy, dw = mx.token_combine_grad(dout, y, w, plan)
    check_gradient(plan, dout, y, w, dy, dw, k, H)


def test_gradient_with_lists_of_entries_out_of_range():
    """An entry out of range counts as absent, and is reported."""
    T, k, H = 9001, 8, 2056
    gen, good = routed(T, k, 64, 8, 4)
    rows = good.src.numel()
    slot, src = good.slot.clone().view(-1), good.src.clone()
    lost = torch.nonzero((torch.rand(rows, generator=gen, device="cuda") < 0.2) & (src >= 0)).squeeze(-1)
    pairs = src[lost].long()
    slot[pairs], src[lost] = -1, -1
    clean = mx.TokenPlan(good.offs, slot.view(T, k), src)
    wild = torch.tensor([rows, rows + 5, 2 ** 31 - 1, -2, -(2 ** 31)], dtype=torch.int32, device="cuda")
    bad_slot, bad_src = slot.clone(), src.clone()
    n = torch.arange(len(lost), device="cuda")
    bad_slot[pairs] = wild[n % 5]
    bad_src[lost] = torch.where(n % 2 == 0, torch.tensor(T * k, dtype=torch.int32, device="cuda"), wild[2 + n % 3])
    bad = mx.TokenPlan(good.offs, bad_slot.view(T, k), bad_src)
    dout, y, w = rand(gen, T, H), rand(gen, rows, H), torch.rand((T, k), generator=gen, device="cuda")
    want = mx.token_combine_grad(dout, y, w, clean)
    assert mx.device_status(clear=True) == 0
    check_gradient(clean, dout, y, w, *want, k, H)
    got = mx.token_combine_grad(dout, y, w, bad)
    assert mx.device_status(clear=True) == _lib.DEV_TOKENS_RANGE
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gradient_with_lists_captured():
    """Replayed on another routing and other values in the same buffers."""
    T, k, H, rows = 9001, 8, 2056, 12800
    sets = []
    for seed in (5, 6):
        gen, plan = routed(T, k, 64, 8, seed, rows=rows)
        sets.append((rand(gen, T, H), rand(gen, rows, H), torch.rand((T, k), generator=gen, device="cuda"), plan.slot, plan.src))
    call = lambda dout, y, w, slot, src: mx.token_combine_grad(dout, y, w, mx.TokenPlan(slot[:1, 0], slot, src))  # noqa: E731
    want = [call(*a) for a in sets]
    live = [a.clone() for a in sets[0]]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(*live)
    for i in (1, 0, 1):
        for a, b in zip(live, sets[i]):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
