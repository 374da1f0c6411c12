"""Outputs that a call allocates itself belong to the stream that writes them.

A tensor allocated on another stream than the one whose kernel writes it may
share its memory with work of the first stream that is still queued, and may be
given away after it is dropped while the kernel still writes. On the CPU: the
calls run on stand-ins (host tensors that pass for CUDA ones, a library that
records and computes nothing), and the stream current at each allocation is
recorded. On the GPU: the allocator's own record of each output's stream."""
import contextlib
import types

import pytest
import torch

import moe_ragged_contraction_gb300 as mx
from moe_ragged_contraction_gb300 import _lib, experts

E, N, K, M, T = 4, 64, 96, 128, 3


def calls(t):
    """name -> call(stream=...) returning the outputs it allocates; t(dtype, *shape) makes an input."""
    u8, bf, f32, i32 = torch.uint8, torch.bfloat16, torch.float32, torch.int32
    A, sA, B, sB, offs = t(u8, N, M), t(u8, N, M // 32), t(u8, K, M), t(u8, K, M // 32), t(i32, E)
    X, sX, W, sW = t(u8, M, K), t(u8, M, K // 32), t(u8, E, N, K), t(u8, E, N, K // 32)
    x16, x32 = t(bf, M, N), t(f32, N, M)
    x, router, w13, s13, w2, s2 = t(bf, T, K), t(bf, E, K), t(u8, E, 2 * N, K), t(u8, E, 2 * N, K // 32), t(u8, E, K, N), t(u8, E, K, N // 32)
    grad = t(bf, E, N, K)
    sfA, sfB = t(u8, 4096), t(u8, 4096)  # (blocks of up to 4 tiles of 256 rows by one 128-token step)
    return {
        "moe_layer": lambda stream: [mx.moe_layer(x, router, w13, s13, w2, s2, 2, stream=stream)],
        "muon_update": lambda stream: [mx.muon_update(grad, stream=stream)],
        "wgrad_grouped": lambda stream: [mx.wgrad_grouped(A, sA, B, sB, offs, stream=stream)],
        "wgrad_grouped_sf": lambda stream: [mx.wgrad_grouped_sf(A, sfA, B, sfB, offs, 0, 64, stream=stream)],
        "grouped_gemm": lambda stream: [mx.grouped_gemm(X, sX, W, sW, offs, stream=stream)],
        "quantize_tokenwise": lambda stream: list(mx.quantize_tokenwise(x32, stream=stream)),
        "quantize_transpose_bf16": lambda stream: list(mx.quantize_transpose_bf16(x16, stream=stream)),
        "quantize_transpose_bf16_sf": lambda stream: list(mx.quantize_transpose_bf16_sf(x16, 64, stream=stream)[:2]),
    }


def names():
    return list(calls(lambda dtype, *shape: None))


class Host(torch.Tensor):
    """A host tensor that passes for one on cuda:0."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cpu"))

    def get_device(self):
        return 0


class Library:
    def __getattr__(self, name):
        return lambda *args: 4096 if name.endswith("bytes") else 0


@pytest.mark.parametrize("name", names())
def test_outputs_are_allocated_under_the_given_stream(monkeypatch, name):
    current, seen = [0], []

    @contextlib.contextmanager
    def under(stream):
        old, current[0] = current[0], stream.cuda_stream
        yield
        current[0] = old

    def recorded(f):
        def g(*a, **kw):
            seen.append(current[0])
            return f(*a, **kw).as_subclass(Host)
        return g

    inputs = calls(lambda dtype, *shape: torch.zeros(shape, dtype=dtype).as_subclass(Host))
    monkeypatch.setattr(_lib, "_lib", Library())
    monkeypatch.setattr(experts, "_torch", torch)
    monkeypatch.setattr(experts, "_raw_stream", lambda device: current[0])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=current[0], device_index=0))
    monkeypatch.setattr(torch.cuda, "stream", under)
    for f in ("empty", "empty_like"):
        monkeypatch.setattr(torch, f, recorded(getattr(torch, f)))
    inputs[name](types.SimpleNamespace(cuda_stream=77, device_index=0))
    assert seen and set(seen) == {77}
    seen.clear()
    inputs[name](None)
    assert seen and set(seen) == {0}


@pytest.mark.gpu
@pytest.mark.parametrize("name", names())
def test_the_allocator_knows_the_stream(name):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.build()
    run = calls(lambda dtype, *shape: torch.zeros(shape, dtype=dtype, device="cuda"))[name]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream, want in ((side, side.cuda_stream), (None, torch.cuda.current_stream().cuda_stream)):
        outs = run(stream)
        torch.cuda.synchronize()
        segments = torch.cuda.memory_snapshot()
        for o in outs:
            p = o.data_ptr()
            assert [s["stream"] for s in segments if s["address"] <= p < s["address"] + s["total_size"]] == [want]
    assert mx.device_status(clear=True) == 0
