"""Shapes with a dimension of 2^31 or more: the library's 32-bit sizes would take it
modulo 2^32 and work on a part of the tensors. On host tensors that pass for CUDA
ones and, being empty in another dimension, hold nothing."""
import pytest
import torch

import moe_ragged_contraction_gb300 as mx
from moe_ragged_contraction_gb300 import _lib, experts

BIG = 2 ** 32
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
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: type("S", (), {"cuda_stream": 0})())
    return names


def plan(k=2):
    return mx.TokenPlan(t(i32, 4), t(i32, 0, k), t(i32, 0))


H = BIG + 64


@pytest.mark.parametrize("call", [
    lambda: mx.token_plan(t(i32, 0, BIG + 2), 4, rows=0, out=mx.TokenPlan(t(i32, 4), t(i32, 0, BIG + 2), t(i32, 0))),
    lambda: mx.token_dispatch(t(bf, 0, H), plan(), out=t(bf, 0, H)),
    lambda: mx.token_dispatch(t(bf, 0, 64), plan(BIG + 2), out=t(bf, 0, 64)),
    lambda: mx.token_dispatch_mxfp8(t(bf, 0, H), plan(), q=t(u8, 0, H), s=t(u8, 0, H // 32)),
    lambda: mx.token_dispatch_grad(t(bf, 0, H), plan(), out=t(bf, 0, H)),
    lambda: mx.token_combine(t(bf, 0, H), t(f32, 0, 2), plan(), out=t(bf, 0, H)),
    lambda: mx.token_combine(t(bf, 0, 64), t(f32, 0, BIG + 2), plan(BIG + 2), out=t(bf, 0, 64)),
    lambda: mx.token_combine_grad(t(bf, 0, H), t(bf, 0, H), t(f32, 0, 2), plan(), dy=t(bf, 0, H), dweights=t(f32, 0, 2)),
    lambda: mx.moe_layer(t(bf, 3, 0), t(bf, BIG + 4, 0), t(u8, 4, 64, 0), t(u8, 4, 64, 0), t(u8, 4, 0, 32), t(u8, 4, 0, 1), 2, out=t(bf, 3, 0)),
    lambda: mx.moe_layer(t(bf, 0, H), t(bf, 0, H), t(u8, 0, 64, H), t(u8, 0, 64, H // 32), t(u8, 0, H, 32), t(u8, 0, H, 1), 2, out=t(bf, 0, H)),
    lambda: mx.moe_layer(t(bf, 0, 0), t(bf, 4, 0), t(u8, 0, 2 * H, 0), t(u8, 0, 2 * H, 0), t(u8, 0, 0, H), t(u8, 0, 0, H // 32), 2, out=t(bf, 0, 0)),
    lambda: mx.muon_update(t(bf, BIG + 1, 0, 8), out=t(bf, BIG + 1, 0, 8)),
    lambda: mx.muon_update(t(bf, 0, BIG + 8, 8), out=t(bf, 0, BIG + 8, 8)),
    lambda: mx.muon_update(t(bf, 0, 8, BIG + 8), out=t(bf, 0, 8, BIG + 8)),
    lambda: mx.wgrad_grouped(t(u8, H, 0), t(u8, H, 0), t(u8, 64, 0), t(u8, 64, 0), t(i32, 0), out=t(bf, 0, H, 64)),
    lambda: mx.wgrad_grouped(t(u8, 64, 0), t(u8, 64, 0), t(u8, H, 0), t(u8, H, 0), t(i32, 0), out=t(bf, 0, 64, H)),
    lambda: mx.wgrad_grouped_sf(t(u8, H, 0), t(u8, 8), t(u8, 64, 0), t(u8, 8), t(i32, 0), 0, 64, out=t(bf, 0, H, 64)),
    lambda: mx.grouped_gemm(t(u8, 0, 32), t(u8, 0, 1), t(u8, 0, H, 32), t(u8, 0, H, 1), t(i32, 0), out=t(bf, 0, H)),
    lambda: mx.quantize_tokenwise(t(f32, H, 0), q=t(u8, H, 0), s=t(u8, H, 0)),
    lambda: mx.quantize_transpose_bf16(t(bf, 0, H), q=t(u8, H, 0), s=t(u8, H, 0)),
])
def test_refused(asked, call):
    with pytest.raises(ValueError):
        call()
    assert not [n for n in asked if not n.endswith("bytes")]


def test_queries(monkeypatch):
    mx.build()
    assert mx.workspace_bytes(4, 128, 64, 256) > 0 and mx.sf_blocks_bytes(128, 256, 64) > 0
    assert mx.workspace_bytes(BIG + 4, 128, 64, 256) == mx.workspace_bytes(4, BIG + 128, 64, 256) == mx.workspace_bytes(4, 128, BIG + 64, 256) == 0
    assert mx.sf_blocks_bytes(BIG + 128, 256, 64) == mx.sf_blocks_bytes(128, 256, BIG + 64) == 0
    for query in (mx.tile_config, mx.grouped_gemm_tile_config):
        assert query(4, 128, 64, 256)
        for sizes in ((BIG + 4, 128, 64, 256), (4, BIG + 128, 64, 256), (4, 128, BIG + 64, 256)):
            with pytest.raises((ValueError, mx.Mxfp8Error)):
                query(*sizes)
