"""moe_layer where tiles are cut along the contraction: eight parts in either
phase, and calls that take the form which can cut where the routing, known on the
GPU only, then leaves nothing to cut. The rules are restated here so that each
case is what it says."""
import numpy as np
import pytest
import torch

import moe_ragged_contraction_gb300 as mx
import oracle
from test_gpu_moe_layer import check, cuda, device_args, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.build()
    oracle.build()
    mx.device_status(clear=True)


def parts(H, I, chosen, sms):
    """(parts of an up/gate tile, of a down tile) with so many chosen experts."""
    up, down, up_steps, down_steps = -(-I // 64), -(-H // 128), -(-H // 128), -(-I // 128)
    of = lambda tiles, steps: 1 if 2 * tiles > sms else max(1, min(sms // max(tiles, 1), steps // 4, 8))  # noqa: E731
    return of(chosen * up, up_steps), of(chosen * down, down_steps)


def can_cut(T, H, I, experts, local, top_k, sms):
    chosen = min(max(T * top_k * local // experts, 1), local)
    return (-(-H // 128) >= 32 and chosen * -(-I // 64) <= sms) or (-(-I // 128) >= 32 and chosen * -(-H // 128) <= sms)


@pytest.mark.parametrize("T,H,I,experts,local,first,top_k,want", [
    (2, 4096, 96, 6, 2, 2, 2, (8, 1)),        # two up/gate tiles an expert, 32 K-steps in 8 parts
    (70, 4128, 64, 6, 2, 2, 2, (8, 1)),       # 33 K-steps; more than 128 columns
    (2, 160, 4128, 6, 2, 2, 2, (1, 8)),       # two down tiles an expert, 33 K-steps in 8 parts
    (1, 4256, 4096, 6, 1, 2, 1, (2, 4)),      # both phases cut, neither in 8
    (1, 4096, 320, 1024, 16, 500, 16, (1, 1)),  # one chosen expert expected here, sixteen chosen: nothing is cut
])
def test_parts(T, H, I, experts, local, first, top_k, want):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert can_cut(T, H, I, experts, local, top_k, sms) and parts(H, I, min(local, top_k), sms) == want
    ops = make(T, H, I, experts, local, seed=H + I)
    bias = np.zeros(experts, np.float32)
    bias[first:first + local] = 9.0 + 0.5 * np.arange(local)  # every token to the experts that live here, far from ties
    args = device_args(*ops)
    out, ids, weights = run(args, top_k, bias=cuda(bias), first_expert=first)
    check(*ops, top_k, out, ids, weights, first=first, bias=bias)
    assert set(ids.cpu().numpy().ravel().tolist()) == set(range(first, first + local))
    again, _, _ = run(args, top_k, bias=cuda(bias), first_expert=first)
    assert torch.equal(out, again)
