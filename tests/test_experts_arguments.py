"""Arguments that the expert-weight operators would take for something else:
inputs that require a gradient (the result would be cut from the graph without
a word) and numbers that do not fit the library's 32-bit integers (they would be
taken modulo 2^32). On host tensors that pass for CUDA ones."""
import types

import numpy as np
import pytest
import torch

import moe_ragged_contraction_gb300 as mx
from moe_ragged_contraction_gb300 import _lib, experts

E, H, I, T = 4, 96, 64, 3


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


def layer(**kw):
    u8, bf = torch.uint8, torch.bfloat16
    args = dict(x=t(bf, T, H), router=t(bf, E, H), w13=t(u8, E, 2 * I, H), s13=t(u8, E, 2 * I, H // 32), w2=t(u8, E, H, I), s2=t(u8, E, H, I // 32),
                top_k=2, bias=t(torch.float32, E))
    args.update(kw)
    return mx.moe_layer(**args)


def update(**kw):
    args = dict(grad=t(torch.float32, E, H, I), momentum=t(torch.float32, E, H, I))
    args.update(kw)
    return mx.muon_update(**args)


@pytest.mark.parametrize("call,name,value", [
    (layer, "x", lambda: t(torch.bfloat16, T, H)), (layer, "router", lambda: t(torch.bfloat16, E, H)), (layer, "bias", lambda: t(torch.float32, E)),
    (layer, "out", lambda: t(torch.bfloat16, T, H)), (layer, "topk_weights", lambda: t(torch.float32, T, 2)),
    (update, "grad", lambda: t(torch.float32, E, H, I)), (update, "momentum", lambda: t(torch.float32, E, H, I)),
    (update, "out", lambda: t(torch.bfloat16, E, H, I)),
])
def test_tensors_that_require_a_gradient(asked, call, name, value):
    v = value().requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        call(**{name: v})
    assert not asked
    with torch.no_grad():
        call(**{name: v})
    call(**{name: v.detach()})
    assert len(asked) == 2


BIG = 2 ** 32


@pytest.mark.parametrize("call,kw", [
    (layer, dict(top_k=BIG + 2)), (layer, dict(first_expert=BIG)), (layer, dict(top_k=2 - BIG)), (layer, dict(first_expert=-BIG)),
    (update, dict(steps=BIG + 5)), (update, dict(steps=5 - BIG)),
])
def test_integers_beyond_32_bits(asked, call, kw):
    with pytest.raises(ValueError):
        call(**kw)
    assert not asked


def test_integers_of_other_kinds(asked):
    layer(top_k=np.int64(2), first_expert=np.int32(0))
    update(steps=np.int64(3))
    assert len(asked) == 2
    with pytest.raises(TypeError):
        layer(top_k=2.0)
    with pytest.raises(TypeError):
        update(steps="5")


def test_workspace_queries_beyond_32_bits():
    mx.build()
    assert mx.moe_layer_workspace_bytes(4, 8, 8, 64, 32, 2) > 0 and mx.muon_update_workspace_bytes(1, 136, 136) > 0
    for bad in ((BIG + 4, 8, 8, 64, 32, 2), (4, 8, 8, 64, BIG + 32, 2), (4, 8, 8, 64, 32, BIG + 2)):
        assert mx.moe_layer_workspace_bytes(*bad) == 0
    for bad in ((BIG + 1, 136, 136), (1, BIG + 136, 136), (1, 136, 136 - BIG)):
        assert mx.muon_update_workspace_bytes(*bad) == 0
