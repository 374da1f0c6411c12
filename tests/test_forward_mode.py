"""Inputs with a forward-mode tangent (torch.autograd.forward_ad): the operators have
no derivative in that direction, and a result without a tangent would be taken for
one that does not depend on the input. On host tensors that pass for CUDA ones."""
import pytest
import torch
import torch.autograd.forward_ad as fwad

import moe_ragged_contraction_gb300 as mx
from moe_ragged_contraction_gb300 import _lib, experts

T, K, H, I, E, ROWS = 6, 2, 64, 32, 3, 96
bf, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


class Host(torch.Tensor):
    """A host tensor that passes for one on cuda:0."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


def t(dtype, *shape):
    return torch.zeros(shape, dtype=dtype).as_subclass(Host)


@pytest.fixture
def asked(monkeypatch):
    """The names of the library's functions that were called; none computes anything."""
    names = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: names.append(name) or 0

    monkeypatch.setattr(_lib, "_lib", Library())
    monkeypatch.setattr(experts, "_torch", torch)
    monkeypatch.setattr(experts, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return names


def arguments():
    plan = mx.TokenPlan(t(i32, E), t(i32, T, K), t(i32, ROWS))
    return {
        "token_dispatch": dict(x=t(bf, T, H), plan=plan, out=t(bf, ROWS, H)),
        "token_dispatch_mxfp8": dict(x=t(bf, T, H), plan=plan, q=t(u8, ROWS, H), s=t(u8, ROWS, H // 32)),
        "token_dispatch_grad": dict(dxs=t(bf, ROWS, H), plan=plan, out=t(bf, T, H)),
        "token_combine": dict(y=t(bf, ROWS, H), weights=t(f32, T, K), plan=plan, out=t(bf, T, H)),
        "token_combine_grad": dict(dout=t(bf, T, H), y=t(bf, ROWS, H), weights=t(f32, T, K), plan=plan, dy=t(bf, ROWS, H), dweights=t(f32, T, K)),
        "grad_norm": dict(grads=[t(bf, 4, 5), t(f32, 7)], out=t(f32)),
        "clip_grads": dict(grads=[t(bf, 4, 5), t(f32, 7)], max_norm=1.0, norm=t(f32), out=[t(bf, 4, 5), t(f32, 7)]),
        "moe_layer": dict(x=t(bf, T, H), router=t(bf, E, H), w13=t(u8, E, 2 * I, H), s13=t(u8, E, 2 * I, H // 32), w2=t(u8, E, H, I), s2=t(u8, E, H, I // 32),
                          top_k=2, bias=t(f32, E), out=t(bf, T, H), topk_weights=t(f32, T, 2)),
        "muon_update": dict(grad=t(f32, E, H, I), momentum=t(f32, E, H, I), out=t(bf, E, H, I)),
    }


CASES = [(op, name, i) for op, args in arguments().items() for name, v in args.items()
         for i, part in enumerate(v if isinstance(v, list) else [v]) if isinstance(part, torch.Tensor) and part.is_floating_point()]


@pytest.mark.parametrize("op,name,i", CASES)
def test_a_tangent_is_refused(asked, op, name, i):
    with fwad.dual_level():
        args = arguments()[op]
        part = args[name][i] if isinstance(args[name], list) else args[name]
        dual = fwad.make_dual(part, torch.ones_like(part))
        assert isinstance(dual, Host) and fwad.unpack_dual(dual).tangent is not None
        changed = {**args, name: args[name][:i] + [dual] + args[name][i + 1:] if isinstance(args[name], list) else dual}
        for context in (torch.enable_grad, torch.no_grad):  # (no_grad does not stop tangents)
            with context(), pytest.raises(ValueError, match=f"{name} has a forward-mode tangent"):
                getattr(mx, op)(**changed)
        assert not asked
        # without the tangent, and others without one
        changed[name] = args[name][:i] + [dual.detach()] + args[name][i + 1:] if isinstance(args[name], list) else dual.detach()
        getattr(mx, op)(**changed)
    assert asked == ["mxfp8_" + op]
