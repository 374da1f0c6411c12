"""One training step of an expert layer, from tokens to updated weights.

  router (torch)             -> ids, weights
  -> token_plan              which row belongs to which (token, expert)
  -> token_dispatch_mxfp8    rows sorted by expert, quantised
  -> grouped_gemm            gate and up, then down
  -> token_combine           the layer's output
  and back: token_combine_grad, the data gradients (grouped_gemm on the
  transposed weights), token_dispatch_grad, the weight gradients
  (quantize_transpose_bf16, wgrad_grouped), then clip_grads and muon_update.

Run on a GB300: python examples/layer_step.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import moe_ragged_contraction_gb300 as mx


def quantised(w):
    """fp32 or bf16 [..., rows, cols] as E4M3 bytes and E8M0 scales along the columns."""
    q, s = mx.quantize_tokenwise(w.float().reshape(-1, w.shape[-1]).contiguous())
    return q.view(w.shape), s.view(*w.shape[:-1], -1)


def layer(x, dout, router, w13, w2, top_k):
    """Output and gradients of the layer for the output gradient dout. x, dout: bf16 [T, H]; router: fp32 [E, H];
    w13: fp32 [E, 2 I, H] (gate rows, then up rows), w2: fp32 [E, H, I]."""
    E, I2, H = w13.shape
    leaf = router.detach().requires_grad_()
    score, ids = torch.topk(x.float() @ leaf.T, top_k)
    soft = torch.softmax(score, -1)
    weights = soft.detach().contiguous()

    plan = mx.token_plan(ids, E)
    xq, xqs = mx.token_dispatch_mxfp8(x, plan)
    gu = mx.grouped_gemm(xq, xqs, *quantised(w13), plan.offs)
    g, u = gu.float().chunk(2, -1)
    sig = torch.sigmoid(g)
    h = (g * sig * u).bfloat16()
    y = mx.grouped_gemm(*quantised(h), *quantised(w2), plan.offs)
    out = mx.token_combine(y, weights, plan)

    dy, dweights = mx.token_combine_grad(dout, y, weights, plan)
    (drouter,) = torch.autograd.grad(soft, leaf, dweights)
    dh = mx.grouped_gemm(*quantised(dy), *quantised(w2.mT.contiguous()), plan.offs).float()
    dgu = torch.cat((dh * u * sig * (1 + g * (1 - sig)), dh * g * sig), -1).bfloat16()
    dxs = mx.grouped_gemm(*quantised(dgu), *quantised(w13.mT.contiguous()), plan.offs)
    dx = mx.token_dispatch_grad(dxs, plan)  # (through the experts; the router's part is torch's)
    xs = mx.token_dispatch(x, plan)
    dw13 = mx.wgrad_grouped(*mx.quantize_transpose_bf16(dgu), *mx.quantize_transpose_bf16(xs), plan.offs)
    dw2 = mx.wgrad_grouped(*mx.quantize_transpose_bf16(dy), *mx.quantize_transpose_bf16(h), plan.offs)
    return out, dx, [dw13, dw2, drouter]


def main(T=1000, E=8, H=512, I=256, top_k=2, lr=0.02, steps=3, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    w13, w2, router = rand(E, 2 * I, H) / H ** 0.5, rand(E, H, I) / I ** 0.5, rand(E, H) / H ** 0.5
    moms = [torch.zeros_like(w13), torch.zeros_like(w2)]
    norms = []
    for _ in range(steps):
        x, dout = rand(T, H).bfloat16(), (rand(T, H) * 0.1).bfloat16()
        out, dx, grads = layer(x, dout, router, w13, w2, top_k)
        norms.append(mx.clip_grads(grads, 1.0))
        for w, mom, g in zip((w13, w2), moms, grads):
            w.add_(mx.muon_update(g, mom), alpha=-lr * 0.02 * max(w.shape[1:]) ** 0.5)
        router.add_(grads[2], alpha=-lr)
    torch.cuda.synchronize()
    if mx.device_status(clear=True):
        raise RuntimeError("a kernel reported an error")
    print(f"{steps} steps of {T} tokens over {E} experts: gradient norms " + ", ".join(f"{float(n):.2f}" for n in norms) + ", clipped to 1")
    return out, norms


if __name__ == "__main__":
    main()
