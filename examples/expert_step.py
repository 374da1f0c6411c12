"""One optimiser step of an expert layer and the next tokens served with it.

The pieces of the package in the order in which a training loop and a server
use them, on synthetic data:

  quantise-and-transpose of the layer's inputs and output gradients
  -> wgrad_grouped      dW of every expert, bf16 [E, N, K]
  -> muon_update        momentum and orthogonalised direction
  -> the caller's step  on fp32 master weights
  -> quantize_tokenwise the updated weights as MXFP8
  -> moe_layer          the layer for a few tokens on the new weights

Run on a GB300: python examples/expert_step.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import moe_ragged_contraction_gb300 as mx


def quantised(w):
    """fp32 weights [E, rows, cols] as E4M3 bytes and E8M0 scales along the columns."""
    E, rows, cols = w.shape
    q, s = mx.quantize_tokenwise(w.reshape(E * rows, cols))
    return q.view(E, rows, cols), s.view(E, rows, cols // 32)


def main(E=8, H=512, I=256, tokens_per_expert=256, top_k=2, lr=0.02, steps=3, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    w13, w2 = rand(E, 2 * I, H) / H ** 0.5, rand(E, H, I) / I ** 0.5  # master weights
    moms = [torch.zeros_like(w13), torch.zeros_like(w2)]
    router = (rand(E, H) / H ** 0.5).bfloat16()
    x = rand(4, H).bfloat16()
    before = mx.moe_layer(x, router, *quantised(w13), *quantised(w2), top_k)

    M = E * tokens_per_expert
    offs = (torch.arange(1, E + 1, dtype=torch.int32, device="cuda") * tokens_per_expert).contiguous()
    offs[2] = offs[1]  # expert 2 gets no tokens (its neighbour takes them): its gradient and update are zero
    for _ in range(steps):
        # token-major bf16 inputs and output gradients of both products, sorted by expert
        for w, mom in ((w13, moms[0]), (w2, moms[1])):
            N, K = w.shape[1:]
            inputs, grads = rand(M, K).bfloat16(), (rand(M, N) * 1e-2).bfloat16()
            A, sA = mx.quantize_transpose_bf16(grads)
            B, sB = mx.quantize_transpose_bf16(inputs)
            dw = mx.wgrad_grouped(A, sA, B, sB, offs)
            update = mx.muon_update(dw, mom)
            # the update's singular values are about one whatever the shape: scale to the weights' spread
            w.add_(update, alpha=-lr * 0.2 * max(N, K) ** 0.5 / 10)
    after = mx.moe_layer(x, router, *quantised(w13), *quantised(w2), top_k)
    torch.cuda.synchronize()
    if mx.device_status(clear=True):
        raise RuntimeError("a kernel reported an error")
    moved = float((after.float() - before.float()).norm() / before.float().norm())
    print(f"{steps} steps over {E} experts of [{2 * I}, {H}] and [{H}, {I}]: the layer's output moved by {moved:.3f} of its norm")
    return before, after, moms, update


if __name__ == "__main__":
    main()
