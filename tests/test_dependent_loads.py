"""What kernels that start as programmatic dependents read. Such a kernel is
resident while the one before it still writes, so ld.global.nc (__ldg), which is
for data that does not change while a kernel runs, could give it lines from
before. On the CPU: the sources hold no such load. On the GPU: gradients clipped in place
and tokens summed up, used by the next call at once, give the bits that they give
with a synchronisation between."""
import os
import re

import pytest
import torch

import moe_ragged_contraction_gb300 as mx

CSRC = os.path.join(os.path.dirname(os.path.abspath(mx.__file__)), "csrc")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


@pytest.mark.parametrize("name", ["muon.cu", "muon_small.cu", "moe_layer.cu", "tokens.cu", "grads.cu"])
def test_no_loads_of_constant_data(name):
    """Sources whose kernels are all launched with the attribute."""
    text = code(name)
    assert "griddep_wait" in text and text.count("__global__") <= text.count("griddep_wait();")
    for word in ("__ldg", "ld.global.nc", "__restrict__"):
        assert word not in text, word


def test_no_loads_of_constant_data_in_the_main_contraction():
    """wgrad_main starts beside the prep kernel that writes its plan. (The prep kernels start after all work before them.)"""
    text = code("wgrad_kernels.cu")
    main = text[text.index("Item load_item("):text.index("long long item_index(")] + text[text.index("struct ItemStream {"):text.index("cudaError_t launch_main(")]
    assert main.count("__global__") == 1 and "griddep_wait();" in main
    for word in ("__ldg", "ld.global.nc", "__restrict__"):
        assert word not in main, word


@pytest.fixture
def rand():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.build()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    yield lambda *shape: torch.randn(shape, generator=gen, device="cuda")
    assert mx.device_status(clear=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(4, 128, 256), (1, 64, 2048), (2, 2048, 128), (3, 264, 520), (2, 1408, 2048), (1, 2048, 1000)])
def test_update_of_gradients_clipped_in_place(rand, shape, dtype):
    """The same buffers hold other gradients at each step; the momentum shows whether the update saw them as clipped."""
    steps = [(rand(*shape) * 2.0 ** k).to(dtype) for k in (3, -2, 5, 0, 4)]
    zeros = [torch.zeros(shape, device="cuda") for _ in range(2)]
    mx.muon_update(steps[0].clone(), torch.zeros_like(zeros[0]))  # (scratch and kernels are there from now on)
    torch.cuda.synchronize()
    results = []
    for momentum, wait in zip(zeros, (True, False)):
        grad, other = torch.empty_like(steps[0]), torch.ones(7, device="cuda")
        kept = []
        for g in steps:
            grad.copy_(g)
            mx.clip_grads([grad, other], 0.5)
            if wait:
                torch.cuda.synchronize()
            update = mx.muon_update(grad, momentum)
            kept += [update, momentum.clone(), grad.clone()]
        torch.cuda.synchronize()
        results.append(kept)
    for a, b in zip(*results):
        assert torch.equal(a, b)
    # what was clipped is what the momentum was made of
    m = torch.zeros(shape, dtype=torch.float64, device="cuda")
    for i in range(len(steps)):
        g = results[1][3 * i + 2].double()
        assert float(g.norm()) <= 0.51
        m = 0.95 * m + g
    # (mu is 0.95 in fp32; a fused multiply-add a step: five roundings of sums below 2.5 in magnitude)
    assert float((results[1][-2].double() - m).abs().max()) <= 5 * 2.5 * 2 * 2.0 ** -24


@pytest.mark.gpu
def test_layer_of_tokens_summed_up_just_before(rand):
    T, E, H, I, k = 24, 8, 512, 256, 2
    w13, s13 = mx.quantize_tokenwise(rand(E * 2 * I, H))
    w2, s2 = mx.quantize_tokenwise(rand(E * H, I))
    weights = (rand(E, H).bfloat16(), w13.view(E, 2 * I, H), s13.view(E, 2 * I, -1), w2.view(E, H, I), s2.view(E, H, -1), k)
    ids = torch.arange(T * k, device="cuda").view(T, k) % 5
    plan = mx.token_plan(ids, 5)
    share = torch.full((T, k), 0.5, device="cuda")
    sets = [rand(plan.src.numel(), H).bfloat16() for _ in range(6)]
    mx.moe_layer(rand(T, H).bfloat16(), *weights)
    torch.cuda.synchronize()
    results = []
    for wait in (True, False):
        x, kept = torch.empty((T, H), dtype=torch.bfloat16, device="cuda"), []
        for y in sets:
            mx.token_combine(y, share, plan, out=x)
            if wait:
                torch.cuda.synchronize()
            kept.append(mx.moe_layer(x, *weights))
        torch.cuda.synchronize()
        results.append(kept)
    for a, b in zip(*results):
        assert torch.equal(a, b)
