"""Measured cases of the expert-weight operators: the orthogonalised update of a
stack of expert gradients (Newton-Schulz products) and the whole expert layer
for a few tokens (router, MXFP8 experts, weighted sum).

``own`` chooses what ``run`` calls: the plain form (elementary torch operations
in fp32, rounded once at the end) or the package's kernels.
"""
import math

import torch

own = False

COEFFS = (3.4445, -4.7750, 2.0315)  # a, b, c of one Newton-Schulz step a X + (b A + c A A) X, A = X X^T
STEPS = 5
MU = 0.95
EPS = 1e-7

_MOE_WEIGHTS = 32 * 3 * 7168 * 2048      # weights of the largest listed layer: the most a drawn one holds
_MUON_FLOPS = 32 * STEPS * (3 * 2048 ** 2 * 7168 + 2048 ** 3)


def _moe(name, T, H, I, experts, first, local, top_k, score, renormalize, scale):
    return {"name": name, "op": "moe", "T": T, "H": H, "I": I, "experts": experts, "first": first, "local": local,
            "top_k": top_k, "score": score, "renormalize": renormalize, "scale": scale}


def _muon(name, E, N, K, dtype, momentum):
    return {"name": name, "op": "muon", "E": E, "N": N, "K": K, "dtype": dtype, "momentum": momentum}


def listed():
    return [
        # the tiny layer (N=128, K=256): launch and hand-over latency only
        _moe("layer tiny, 1 token", 1, 256, 128, 4, 0, 4, 2, "softmax", True, 1.0),
        # 16B expert shape, all 64 experts of a layer on the card: one sequence decoding
        _moe("layer 16B, 1 token", 1, 2048, 1408, 64, 0, 64, 6, "softmax", False, 1.0),
        # the same layer, a small batch decoding
        _moe("layer 16B, 8 tokens", 8, 2048, 1408, 64, 0, 64, 6, "softmax", False, 1.0),
        # the same layer, a batch that reaches every expert
        _moe("layer 16B, 64 tokens", 64, 2048, 1408, 64, 0, 64, 6, "softmax", False, 1.0),
        # 671B expert shape, the 32 experts of one rank out of 256, sigmoid scores with a selection bias
        _moe("layer 671B rank, 16 tokens", 16, 7168, 2048, 256, 96, 32, 8, "sigmoid", True, 2.5),
        # the same rank with the most tokens a call takes
        _moe("layer 671B rank, 128 tokens", 128, 7168, 2048, 256, 96, 32, 8, "sigmoid", True, 2.5),
        # sizes that fill no tile, a slice of an odd number of experts: many tokens with no local expert
        _moe("layer odd sizes, 5 tokens", 5, 1056, 352, 21, 4, 13, 3, "sigmoid", False, 1.0),
        # the tiny gradient (E=4, N=128, K=256), one expert without tokens
        _muon("update tiny", 4, 128, 256, "bfloat16", True),
        # 16B expert shape, one rank's 8 experts: the usual step
        _muon("update 16B", 8, 1408, 2048, "bfloat16", True),
        # 671B down shape (tall matrices), one rank's 32 experts: the largest
        _muon("update 671B down", 32, 7168, 2048, "bfloat16", True),
        # one accumulated fp32 gradient of a dense matrix, no momentum kept here
        _muon("orthogonalise 2048 x 1408 fp32", 1, 2048, 1408, "float32", False),
        # rows that fill no tile, fp32
        _muon("orthogonalise 3 x 331 x 1000 fp32", 3, 331, 1000, "float32", False),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def _blocks(rng, lo, hi):
    """A count of blocks between lo and hi: odd half of the time (the last tile is then partial), else a multiple of 20."""
    n = _log(rng, lo, hi)
    return min(hi, round(n) | 1) if rng.random() < 0.5 or n < 20 else 20 * min(hi // 20, round(n / 20))


def draw(rng):
    if rng.random() < 0.5:
        T = max(1, min(128, round(_log(rng, 0.7, 130))))
        H = 32 * _blocks(rng, 8, 224)
        I = 32 * _blocks(rng, 4, 64)
        fit = max(1, _MOE_WEIGHTS // (3 * H * I))
        local = max(1, min(fit, 160, round(_log(rng, 1, 160))))
        experts = min(320, round(local * rng.choice((1, 1, 1.5, 2, 4, 8))))
        first = rng.randint(0, experts - local)
        top_k = rng.randint(1, min(8, experts))
        score = rng.choice(("softmax", "sigmoid"))
        c = _moe("", T, H, I, experts, first, local, top_k, score, rng.random() < 0.5, rng.choice((1.0, 2.5)))
    else:
        while True:
            E = max(1, min(32, round(_log(rng, 0.8, 32))))
            N = round(_log(rng, 33, 7168)) | 1
            K = 8 * _blocks(rng, 5, 896)
            m, n = min(N, K), max(N, K)
            if E * STEPS * (3 * m * m * n + m ** 3) <= _MUON_FLOPS and E * N * K <= 32 * 7168 * 2048:
                break
        c = _muon("", E, N, K, rng.choice(("bfloat16", "bfloat16", "float32")), rng.random() < 0.7)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)
    return g


def _mx_weights(gen, E, rows, cols, std):
    """E4M3 bytes [E, rows, cols] and E8M0 scales [E, rows, cols/32] of normal weights whose spread differs by row;
    the smallest power of two that brings a block's largest element to 448 or below is its scale."""
    q = torch.empty((E, rows, cols), dtype=torch.uint8, device="cuda")
    s = torch.empty((E, rows, cols // 32), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (rows * cols))
    for e in range(0, E, step):
        k = min(step, E - e)
        w = torch.randn((k, rows, cols // 32, 32), generator=gen, device="cuda")
        w *= std * torch.exp(0.5 * torch.randn((k, rows, 1, 1), generator=gen, device="cuda"))
        p = torch.ceil(torch.log2(w.abs().amax(-1, keepdim=True) / 448.0)).clamp(-127, 127)
        w = (w * torch.exp2(-p)).clamp(-448.0, 448.0)
        q[e:e + k] = w.to(torch.float8_e4m3fn).view(torch.uint8).view(k, rows, cols)
        s[e:e + k] = (p.squeeze(-1) + 127).to(torch.uint8)
    return q, s


def prepare(case, seed):
    gen = _generator(seed)
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    c = dict(case)
    if c["op"] == "moe":
        T, H, I = c["T"], c["H"], c["I"]
        x = rand(T, H)
        x[:, torch.randint(0, H, (4,), generator=gen, device="cuda")] *= 8.0  # a few strong channels, as hidden states have
        x /= x.square().mean(-1, keepdim=True).sqrt()
        w13, s13 = _mx_weights(gen, c["local"], 2 * I, H, 1.2 / math.sqrt(H))
        w2, s2 = _mx_weights(gen, c["local"], H, I, 1.2 / math.sqrt(I))
        return {"case": c, "x": x.bfloat16(), "router": (rand(c["experts"], H) * (1.6 / math.sqrt(H))).bfloat16(),
                "bias": rand(c["experts"]) * 0.02 if c["score"] == "sigmoid" else None,
                "w13": w13, "s13": s13, "w2": w2, "s2": s2}
    E, N, K = c["E"], c["N"], c["K"]
    # a few strong directions over a noise floor whose rows differ in strength, as the gradients of a layer have
    def gradient():
        g = rand(E, N, K) * torch.exp(0.5 * rand(E, N, 1))
        g += torch.bmm(rand(E, N, 6), rand(E, 6, K))
        g *= 1e-3
        if E >= 4:
            g[1] = 0  # an expert that got no tokens
        return g
    g = gradient().to(getattr(torch, c["dtype"]))
    mom = gradient() * 8.0 if c["momentum"] else None
    return {"case": c, "grad": g, "momentum": mom}


# ------------------------------------------------------------------ one pass

def _decode(q, s):
    """MXFP8 bytes and block scales as fp32 values."""
    v = q.view(torch.float8_e4m3fn).float().view(*s.shape, 32) * torch.exp2(s.float() - 127.0).unsqueeze(-1)
    return v.view(q.shape)


def _plain_moe(st):
    c, x = st["case"], st["x"].float()
    logits = x @ st["router"].float().t()
    if c["score"] == "softmax":
        e = torch.exp(logits - logits.amax(-1, keepdim=True))
        score = e / e.sum(-1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-logits))
    choice = score if st["bias"] is None else score + st["bias"]
    ids = torch.sort(choice, dim=-1, descending=True, stable=True).indices[:, :c["top_k"]]
    w = torch.gather(score, 1, ids)
    if c["renormalize"]:
        w = w / w.sum(-1, keepdim=True)
    dense = torch.zeros_like(score).scatter_(1, ids, w * c["scale"])
    dense = dense[:, c["first"]:c["first"] + c["local"]]                     # [T, local]
    gu = torch.matmul(_decode(st["w13"], st["s13"]), x.t())                  # [local, 2I, T]
    g, u = gu[:, :c["I"]], gu[:, c["I"]:]
    h = g / (1.0 + torch.exp(-g)) * u * dense.t().unsqueeze(1)               # [local, I, T]
    w2 = _decode(st["w2"], st["s2"])
    return torch.matmul(w2, h).sum(0).t().to(torch.bfloat16)


def _plain_muon(st):
    u = st["grad"].float()
    mom = st["momentum"]
    if mom is not None:
        mom.mul_(MU).add_(u)
        u = u + MU * mom
    X = u / (u.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    tall = X.shape[1] > X.shape[2]
    if tall:
        X = X.mT
    a, b, c = COEFFS
    for _ in range(STEPS):
        A = X @ X.mT
        X = a * X + (b * A + c * (A @ A)) @ X
    if tall:
        X = X.mT
    return X.to(torch.bfloat16).contiguous()


def run(state):
    c = state["case"]
    if c["op"] == "moe":
        if not own:
            return _plain_moe(state)
        import moe_ragged_contraction_gb300 as mx

        return mx.moe_layer(state["x"], state["router"], state["w13"], state["s13"], state["w2"], state["s2"], c["top_k"],
                            bias=state["bias"], first_expert=c["first"], score=c["score"], renormalize=c["renormalize"],
                            scale=c["scale"])
    mom = state["momentum"]
    if own:
        import moe_ragged_contraction_gb300 as mx

        update = mx.muon_update(state["grad"], mom, mu=MU, nesterov=True, steps=STEPS, coeffs=COEFFS, eps=EPS)
    else:
        update = _plain_muon(state)
    return update if mom is None else (update, mom)


def work(case):
    c = case
    if c["op"] == "moe":
        T, H, I = c["T"], c["H"], c["I"]
        touched = c["local"] * (1.0 - (1.0 - c["top_k"] / c["experts"]) ** T)  # experts that some token chose, expected
        weights = touched * 3 * H * I * 33 / 32
        pairs = T * c["top_k"] * c["local"] / c["experts"]
        return {"bytes": weights + 2 * c["experts"] * H + 4 * T * H, "flops": 6 * pairs * H * I + 2 * T * c["experts"] * H}
    size = c["E"] * c["N"] * c["K"]
    m, n = min(c["N"], c["K"]), max(c["N"], c["K"])
    item = 2 if c["dtype"] == "bfloat16" else 4
    # X X^T and A A are symmetric: half of each is enough
    return {"bytes": size * (item + 2 + (8 if c["momentum"] else 0)), "flops": c["E"] * STEPS * (3 * m * m * n + m ** 3)}


# ------------------------------------------------------------------ from the definition, in 64 bits

def _table():
    """The 256 values of E4M3: sign, four exponent bits (bias 7), three fraction bits, no infinities."""
    t = []
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        v = f / 8.0 * 2.0 ** -6 if e == 0 else (1 + f / 8.0) * 2.0 ** (e - 7)
        v = math.nan if e == 15 and f == 7 else v
        t.append(-v if b & 128 else v)
    return torch.tensor(t, dtype=torch.float64, device="cuda")


def _exact_moe(c, st):
    table = _table()

    def matrix(q, s):
        p = torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), s.to(torch.int32) - 127)
        return table[q.long()] * torch.repeat_interleave(p, 32, dim=-1)

    x, R = st["x"].double(), st["router"].double()
    T, k = c["T"], c["top_k"]
    logits = torch.einsum("th,eh->te", x, R).cpu()
    score = torch.softmax(logits, -1) if c["score"] == "softmax" else torch.sigmoid(logits)
    choice = score + (0 if st["bias"] is None else st["bias"].double().cpu())
    chosen = [[] for _ in range(c["local"])]  # per local expert: (token, weight)
    for t in range(T):
        ids = sorted(range(c["experts"]), key=lambda e: (-float(choice[t, e]), e))[:k]
        total = sum(float(score[t, e]) for e in ids) if c["renormalize"] else 1.0
        for e in ids:
            if 0 <= e - c["first"] < c["local"]:
                chosen[e - c["first"]].append((t, float(score[t, e]) / total * c["scale"]))
    y = torch.zeros((T, c["H"]), dtype=torch.float64, device="cuda")
    for e, pairs in enumerate(chosen):
        if pairs:
            at = torch.tensor([t for t, _ in pairs], device="cuda")
            w = torch.tensor([v for _, v in pairs], dtype=torch.float64, device="cuda")
            gu = x[at] @ matrix(st["w13"][e], st["s13"][e]).T
            h = torch.nn.functional.silu(gu[:, :c["I"]]) * gu[:, c["I"]:]
            y.index_add_(0, at, w[:, None] * (h @ matrix(st["w2"][e], st["s2"][e]).T))
    return y


def _exact_muon(c, st):
    a, b, cc = COEFFS
    g = st["grad"].double()
    mom = None if st["momentum"] is None else MU * st["momentum"].double() + g
    out = torch.empty_like(g)
    eye = torch.eye(min(c["N"], c["K"]), dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        u = g[e] if mom is None else g[e] + MU * mom[e]
        X = u / (torch.linalg.vector_norm(u) + EPS)
        for _ in range(STEPS):  # X p(X^T X) on the shorter side
            if c["N"] <= c["K"]:
                A = X @ X.T
                X = (a * eye + b * A + cc * (A @ A)) @ X
            else:
                A = X.T @ X
                X = X @ (a * eye + b * A + cc * (A @ A))
        out[e] = X
    return out if mom is None else (out, mom)


def exact(case, seed):
    c = dict(case)
    if c["op"] == "moe":
        return _exact_moe(c, prepare(case, seed))
    m, n = min(c["N"], c["K"]), max(c["N"], c["K"])
    if c["E"] * STEPS * (4 * m * m * n + 2 * m ** 3) > 8e12:  # 64-bit products of this size take too long
        return None
    return _exact_muon(c, prepare(case, seed))
