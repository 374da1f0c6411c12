"""Measured cases of the operators around the expert products of a training
step: tokens sorted by expert and back (with the router's weights, and both
gradients), and the global norm and clipping of the gradients.

``own`` chooses what ``run`` calls: the plain form (elementary torch operations
in fp32, long sums in fp64, rounded once at the end) or the package's kernels.
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6

_PAIRS_H = 16384 * 6 * 2048          # pairs times columns of the listed 16B cases: the most that a drawn case has
_ELEMENTS = 6 * 8 * 3 * 1408 * 2048  # elements of the largest listed list of gradients


def _tokens(name, op, T, H, experts, first, local, top_k, align=32, spare=0.0, mxfp8=False, padded=0, ids="int32"):
    """spare: 0 for rows that hold every routing, else the share over the expected number of pairs."""
    return {"name": name, "op": op, "T": T, "H": H, "experts": experts, "first": first, "local": local, "top_k": top_k,
            "align": align, "spare": spare, "mxfp8": mxfp8, "padded": padded, "ids": ids}


def _grads(name, op, tensors, total, sizes, dtype, flat=False, clipped=False, out=False):
    """sizes: "stack" (pairs of expert stacks in the ratio 2 : 1 and a small router each) or a seed of mixed sizes."""
    return {"name": name, "op": op, "tensors": tensors, "total": total, "sizes": sizes, "dtype": dtype, "flat": flat,
            "clipped": clipped, "out": out}


def listed():
    return [
        # the tiny layer (4 experts, 256 columns), one token: launches only
        _tokens("dispatch tiny, 1 token", "dispatch", 1, 256, 4, 0, 4, 2),
        # 16B expert shape, all 64 experts here, the tokens of one training micro-batch
        _tokens("dispatch 16B", "dispatch", 16384, 2048, 64, 0, 64, 6),
        # 671B expert shape, one rank's 32 of 256 experts, rows for half as many pairs again as expected, straight to MXFP8
        _tokens("dispatch 671B rank, MXFP8", "dispatch", 32768, 7168, 256, 96, 32, 8, spare=0.5, mxfp8=True),
        # the gradient of the tokens of the 16B micro-batch
        _tokens("dispatch grad 16B", "dispatch_grad", 16384, 2048, 64, 0, 64, 6),
        # sizes that fill no block, any row boundaries, a padded batch: 100 tokens without experts
        _tokens("dispatch grad odd sizes", "dispatch_grad", 1021, 1096, 21, 4, 13, 3, align=1, padded=100),
        # a prompt of a few tokens on one rank: latency
        _tokens("combine 671B rank, 8 tokens", "combine", 8, 7168, 256, 96, 32, 8),
        # the 16B micro-batch back in token order
        _tokens("combine 16B", "combine", 16384, 2048, 64, 0, 64, 6),
        # sizes that fill no block, many tokens without a pair here, a padded batch
        _tokens("combine grad odd sizes", "combine_grad", 1021, 1096, 21, 4, 13, 3, padded=100),
        # one rank's share of the gradient, with the gradient of the router's weights
        _tokens("combine grad 671B rank", "combine_grad", 32768, 7168, 256, 96, 32, 8, spare=0.5),
        # many tensors of a model, small and large, views of one flat buffer
        _grads("norm of 300 tensors, flat", "norm", 300, 40_000_000, "7", "float32", flat=True),
        # the gradients of the tiny layer, within the limit: nothing to scale
        _grads("clip tiny", "clip", 3, 4 * 3 * 128 * 256 + 4 * 256, "stack", "bfloat16"),
        # bf16 gradients of six 16B layers (8 experts each), over the limit, kept beside the clipped ones
        _grads("clip 16B, 6 layers", "clip", 18, _ELEMENTS + 6 * 64 * 2048, "stack", "bfloat16", clipped=True, out=True),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def draw(rng):
    if rng.random() < 0.7:
        op = rng.choice(("dispatch", "dispatch", "dispatch_grad", "combine", "combine_grad"))
        mxfp8 = op == "dispatch" and rng.random() < 0.5
        unit = 32 if mxfp8 else 8
        H = unit * max(1, round(_log(rng, 64, 7168) / unit))
        top_k = rng.randint(1, 8)
        most = max(1, _PAIRS_H // (top_k * H))
        T = max(1, min(most, round(_log(rng, 0.7, min(65536, 1.3 * most)))))
        local = max(1, min(160, round(_log(rng, 1, 160))))
        experts = max(top_k, round(local * rng.choice((1, 1, 1.5, 2, 4, 8))))
        first = rng.randint(0, experts - local)
        spare = rng.choice((0.0, 0.0, 1.0)) if experts >= 2 * local and T >= 256 else 0.0
        c = _tokens("", op, T, H, experts, first, local, top_k, rng.choice((1, 32, 32, 32, 128)), spare, mxfp8,
                    rng.choice((0, T // 10)), rng.choice(("int32", "int64")))
    else:
        op = rng.choice(("norm", "clip", "clip"))
        tensors = max(1, min(60 if op == "clip" else 1500, round(_log(rng, 0.8, 60 if op == "clip" else 1500))))
        total = max(4 * tensors, round(_log(rng, 50, _ELEMENTS / 2))) | 1
        clipped = op == "clip" and rng.random() < 0.7
        c = _grads("", op, tensors, total, str(rng.randint(1, 10 ** 6)), rng.choice(("bfloat16", "float32", "mixed")),
                   rng.random() < 0.5, clipped, clipped)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 29)
    return g


def _rows(c):
    """Rows of the sorted buffers: enough for every routing, or (one rank of several) for `spare` more than expected."""
    pairs, a = c["T"] * c["top_k"], c["align"]
    every = (pairs + min(c["local"], pairs) * (a - 1)) // a * a
    if not c["spare"]:
        return every
    expected = pairs * c["local"] / c["experts"]
    return min(every, (math.ceil(expected * (1 + c["spare"]) + c["local"] * a + 64) + a - 1) // a * a)


def _sizes(c):
    n, total = c["tensors"], c["total"]
    if c["sizes"] == "stack":
        small = 4 * 256 if total < 10 ** 6 else 64 * 2048
        part = (total - n // 3 * small) // (n // 3 * 3)
        return [2 * part, part, small] * (n // 3)
    r = random.Random(int(c["sizes"]))
    raw = [_log(r, 1, 1e4) for _ in range(n)]
    k = total / sum(raw)
    return [max(1, round(v * k)) for v in raw]


def prepare(case, seed):
    gen = _generator(seed)
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    c = dict(case)
    if c["op"] in ("norm", "clip"):
        sizes = _sizes(c)
        types = [torch.float32 if c["dtype"] == "float32" or (c["dtype"] == "mixed" and i % 3 == 2) else torch.bfloat16
                 for i in range(len(sizes))]
        grads = [None] * len(sizes)
        for t in (torch.bfloat16, torch.float32):
            mine = [i for i in range(len(sizes)) if types[i] is t]
            flat = torch.empty(sum(sizes[i] for i in mine) if c["flat"] else 0, dtype=t, device="cuda")
            at = 0
            for i in mine:
                # tensors of different strength, a few strong elements in each, as the gradients of a model have
                g = rand(sizes[i]).mul_(1e-3 * math.exp(1.5 * math.sin(i + 1.0)))
                g[::997] *= 16.0
                if c["flat"]:
                    grads[i] = flat[at:at + sizes[i]]
                    grads[i].copy_(g)
                    at += sizes[i]
                else:
                    grads[i] = g.to(t)
        typical = 1e-3 * 2.0 * math.sqrt(sum(sizes))
        return {"case": c, "grads": grads, "max_norm": typical * (0.0625 if c["clipped"] else 16.0),
                "out": [torch.empty_like(g) for g in grads] if c["out"] else None}
    T, H, k = c["T"], c["H"], c["top_k"]
    logits = rand(T, c["experts"]) + 0.4 * rand(c["experts"])  # some experts are busier than others
    top = torch.topk(logits, k)
    weights, ids = torch.softmax(top.values, -1), top.indices.to(getattr(torch, c["ids"]))
    if c["padded"]:
        ids[T - c["padded"]:] = -1
    st = {"case": c, "ids": ids.contiguous(), "rows": _rows(c)}
    if c["op"] == "dispatch":
        x = rand(T, H)
        x[:, torch.randint(0, H, (4,), generator=gen, device="cuda")] *= 8.0  # a few strong channels, as hidden states have
        st["x"] = x.bfloat16()
        return st
    st["plan"] = _plain_plan(st)
    y = torch.empty((st["rows"], H), dtype=torch.bfloat16, device="cuda")
    step = max(1, (1 << 26) // H)
    for r in range(0, st["rows"], step):
        n = min(step, st["rows"] - r)
        y[r:r + n] = rand(n, H) * torch.exp(0.5 * rand(n, 1))
    st["y"] = y
    if c["op"] != "dispatch_grad":
        st["weights"] = weights.contiguous()
    if c["op"] == "combine_grad":
        st["dout"] = (rand(T, H) * 1e-2).bfloat16()
    return st


# ------------------------------------------------------------------ one pass

def _plain_plan(st):
    """(offs, slot, src): group ends, the row of each (token, choice) pair or -1, the pair of each row or -1."""
    c, rows = st["case"], st["rows"]
    local, a = c["local"], c["align"]
    e = st["ids"].long().reshape(-1) - c["first"]
    key = torch.where((e >= 0) & (e < local), e, local)
    count = torch.zeros(local + 1, dtype=torch.int64, device=key.device).scatter_add_(0, key, torch.ones_like(key))
    ends = torch.cumsum((count[:local] + (a - 1)) // a * a, 0)
    base = torch.cat((ends - (count[:local] + (a - 1)) // a * a, ends.new_zeros(1)))
    before = torch.cumsum(count, 0) - count                        # pairs of lower experts
    order = torch.sort(key, stable=True).indices
    sorted_key = key[order]
    row = base[sorted_key] + torch.arange(key.numel(), device=key.device) - before[sorted_key]
    row = torch.where((sorted_key < local) & (row < rows), row, -1)
    slot = torch.empty_like(key).scatter_(0, order, row)
    src = torch.full((rows + 1,), -1, dtype=torch.int64, device=key.device)
    src.scatter_(0, torch.where(row >= 0, row, rows), order)       # (absent pairs go to a row that is cut off)
    return (ends.clamp(max=rows).to(torch.int32), slot.view(c["T"], c["top_k"]).to(torch.int32), src[:rows].to(torch.int32))


def _plain_dispatch(st):
    c, x = st["case"], st["x"]
    plan = _plain_plan(st)
    src = plan[2].long()
    at = torch.where(src >= 0, src // c["top_k"], c["T"])
    if not c["mxfp8"]:
        xs = torch.cat((x, x.new_zeros(1, c["H"])))[at]
        return plan + (xs,)
    v = x.float().view(c["T"], c["H"] // 32, 32)
    m, p = torch.frexp(v.abs().amax(-1, keepdim=True).double() / 448.0)
    p = torch.where(m == 0, -127, p - (m == 0.5).to(p.dtype)).clamp(-127, 127)  # the smallest power with amax <= 448 * 2^p
    q = (v * torch.exp2(-p.float())).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8).view(c["T"], c["H"])
    s = (p.squeeze(-1) + 127).to(torch.uint8)
    q = torch.cat((q, q.new_zeros(1, c["H"])))[at]
    s = torch.cat((s, s.new_zeros(1, c["H"] // 32)))[at]
    return plan + (q.view(torch.float8_e4m3fn), s)


def _gathered(y, slot):
    """Rows slot of y in fp32, zeros where slot is -1."""
    return torch.where((slot >= 0).unsqueeze(-1), y[slot.clamp(min=0).long()].float(), 0.0)


def _plain_combine(st):
    slot, w = st["plan"][1], st.get("weights")
    acc = torch.zeros((st["case"]["T"], st["case"]["H"]), device=slot.device)
    for j in range(st["case"]["top_k"]):
        rows = _gathered(st["y"], slot[:, j])
        acc += rows if w is None else rows * torch.where(slot[:, j] >= 0, w[:, j], 0.0).unsqueeze(-1)
    return acc.to(torch.bfloat16)


def _plain_combine_grad(st):
    (_, slot, src), k = st["plan"], st["case"]["top_k"]
    dout = st["dout"].float()
    dw = torch.stack([(_gathered(st["y"], slot[:, j]) * dout).sum(-1) for j in range(k)], 1)
    p = src.clamp(min=0).long()
    w = torch.where(src >= 0, st["weights"].reshape(-1)[p], 0.0)
    return (dout[p // k] * w.unsqueeze(-1)).to(torch.bfloat16), dw


def _plain_norm(grads):
    return sum(g.double().square().sum() for g in grads).sqrt()


def _plain_clip(st):
    norm = _plain_norm(st["grads"])
    c = (st["max_norm"] / (norm + EPS)).clamp(max=1.0)
    to = st["out"] if st["case"]["out"] else st["grads"]
    return norm.float(), [o.copy_(g.float() * c.float()) for g, o in zip(st["grads"], to)]


def _own(state):
    import moe_ragged_contraction_gb300 as mx

    c = state["case"]
    if c["op"] == "dispatch":
        plan = mx.token_plan(state["ids"], c["local"], first_expert=c["first"], align=c["align"], rows=state["rows"])
        if not c["mxfp8"]:
            return (*plan, mx.token_dispatch(state["x"], plan))
        q, s = mx.token_dispatch_mxfp8(state["x"], plan)
        return (*plan, q.view(torch.float8_e4m3fn), s)
    if c["op"] == "norm":
        return mx.grad_norm(state["grads"])
    if c["op"] == "clip":
        norm = mx.clip_grads(state["grads"], state["max_norm"], eps=EPS, out=state["out"])
        return norm, state["out"] if c["out"] else state["grads"]
    plan = mx.TokenPlan(*state["plan"])
    if c["op"] == "dispatch_grad":
        return mx.token_dispatch_grad(state["y"], plan)
    if c["op"] == "combine":
        return mx.token_combine(state["y"], state["weights"], plan)
    return mx.token_combine_grad(state["dout"], state["y"], state["weights"], plan)


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "dispatch":
        return _plain_dispatch(state)
    if op == "combine_grad":
        return _plain_combine_grad(state)
    if op == "norm":
        return _plain_norm(state["grads"]).float()
    if op == "clip":
        return _plain_clip(state)
    return _plain_combine(state)


def work(case):
    c = case
    if c["op"] in ("norm", "clip"):
        sizes = _sizes(c)
        item = [4 if c["dtype"] == "float32" or (c["dtype"] == "mixed" and i % 3 == 2) else 2 for i in range(len(sizes))]
        n = sum(a * b for a, b in zip(sizes, item))
        return {"bytes": n * (2 if c["out"] else 1) + 4, "flops": 3 * sum(sizes)}
    T, H, k, rows = c["T"], c["H"], c["top_k"], _rows(c)
    here = c["local"] / c["experts"]
    real = T - c["padded"]
    pairs, tokens = real * k * here, real * (1.0 - (1.0 - here) ** k)  # expected pairs here, tokens with one
    if c["op"] == "dispatch":
        plan = T * k * (8 if c["ids"] == "int64" else 4) + 4 * (T * k + rows + c["local"])
        return {"bytes": plan + 2 * H * tokens + rows * (33 * H / 32 if c["mxfp8"] else 2 * H), "flops": 0}
    if c["op"] == "combine_grad":
        return {"bytes": 2 * H * (tokens + pairs + rows) + 4 * (3 * T * k + rows), "flops": 3 * pairs * H}
    return {"bytes": 2 * H * (pairs + T) + 4 * T * k * (1 if c["op"] == "dispatch_grad" else 2), "flops": 2 * pairs * H}


# ------------------------------------------------------------------ from the definition, in 64 bits

def _exact_plan(c, ids, rows):
    """Expert by expert, in numpy."""
    pairs = ids.cpu().numpy().reshape(-1).astype(np.int64)
    offs, slot, src = np.zeros(c["local"], np.int64), np.full(pairs.size, -1), np.full(rows, -1)
    end = 0
    for e in range(c["local"]):
        mine = np.flatnonzero(pairs == c["first"] + e)
        at = end + np.arange(mine.size)
        fits = at < rows
        slot[mine[fits]], src[at[fits]] = at[fits], mine[fits]
        end += -(-mine.size // c["align"]) * c["align"]
        offs[e] = min(end, rows)
    return offs, slot.reshape(ids.shape), src


def _exact_tokens(c, st):
    k = c["top_k"]
    offs, slot, src = (torch.from_numpy(v).cuda() for v in _exact_plan(c, st["ids"], st["rows"]))
    if c["op"] == "dispatch":
        x = st["x"].double()
        xs = torch.zeros((st["rows"], c["H"]), dtype=torch.float64, device="cuda")
        xs[src >= 0] = x[src[src >= 0] // k]
        ints = (offs.int(), slot.int(), src.int())
        if not c["mxfp8"]:
            return ints + (xs,)
        blocks = xs.view(st["rows"], -1, 32)
        amax = blocks.abs().amax(-1)
        power = torch.full_like(amax, -127.0)
        some = amax > 0
        power[some] = torch.ceil(torch.log2(amax[some] / 448.0)).clamp(-127, 127)  # (bf16 quotients are no nearer to a power of two than 2^-9, or are one)
        return ints + ((blocks / torch.exp2(power)[..., None]).view(xs.shape), (power + 127).to(torch.uint8))
    y = st["y"].double()
    pair = torch.nonzero(slot.reshape(-1) >= 0).squeeze(-1)
    row, token = slot.reshape(-1)[pair], pair // k
    if c["op"] == "combine_grad":
        dout, w = st["dout"].double(), st["weights"].double().reshape(-1)
        dw = torch.zeros_like(w)
        dy = torch.zeros_like(y)
        dw[pair] = torch.einsum("ph,ph->p", y[row], dout[token])
        dy[row] = w[pair, None] * dout[token]
        return dy, dw.view(c["T"], k)
    rows = y[row]
    if c["op"] == "combine":
        rows *= st["weights"].double().reshape(-1)[pair, None]
    out = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device="cuda")
    return out.index_add_(0, token, rows)


def exact(case, seed):
    c = dict(case)
    st = prepare(case, seed)
    if c["op"] not in ("norm", "clip"):
        return _exact_tokens(c, st)
    norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in st["grads"]))
    value = torch.tensor(norm, dtype=torch.float64, device="cuda")
    if c["op"] == "norm":
        return value
    f = min(1.0, st["max_norm"] / (norm + EPS))
    return value, [g.double() * f for g in st["grads"]]
