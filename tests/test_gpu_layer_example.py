"""The decoder layer example runs the operators beside the linears together and
agrees with its own 64-bit form.

Activations are quantised to E4M3 (half a step: 2^-4 of a value at most, 2^-5.5
root mean square over a uniform spread) before each of the products that the
reference takes unquantised -- QKV, output, gate and up, down -- so the residual,
which passes two of them and is dominated by what it was, stays within 2^-4 and
the experts' output, which passes all four and a product of two sums, within
2^-2."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

import block_wise_fp8_gb300 as fb  # noqa: E402
import decoder_layer  # noqa: E402
from test_gpu_lora import reference as lora_reference  # noqa: E402


@pytest.mark.parametrize("M", [1, 5, 33, 64])
def test_decoder_layer(M):
    layer = decoder_layer.Layer(M, H=1024, heads=8, kv_heads=2, D=128, E=16, I=256, topk=4,
                                adapters=4, rank=24, context=31)
    args = decoder_layer.inputs(layer, seed=M, adapters=4)
    y, r = layer.step(*args)
    for ws in (layer.ws_moe, layer.ws_lora, layer.ws_o, layer.ws_qkv):
        assert fb.fp8bq_poll_status(ws) == 0
    ry, rr = layer.reference(*args)
    assert float((r.double() - rr).norm() / rr.norm()) < 2.0 ** -4
    assert float((y.double() - ry).norm() / ry.norm()) < 2.0 ** -2
    first = y.clone()
    assert torch.equal(layer.step(*args)[0], first)


@pytest.mark.parametrize("M", [1, 5, 33, 64])
def test_adapters_within_the_step(M):
    """What each adapter call of a step adds to its projection is the adapters'
    product of that step's own rows, within the bound of that call's own tests."""
    layer = decoder_layer.Layer(M, H=1024, heads=8, kv_heads=2, D=128, E=16, I=256, topk=4,
                                adapters=4, rank=24, context=31)
    calls = []
    add = layer._adapters

    def watched(x, lora, y):
        x0, y0 = x.clone(), y.clone()
        add(x, lora, y)
        calls.append((x0, lora, y0, y.clone()))

    layer._adapters = watched
    args = decoder_layer.inputs(layer, seed=M, adapters=4)
    ids = args[3]
    some = [3, -1, 0, 1, 2][:M]
    ids[:len(some)] = torch.tensor(some, device="cuda", dtype=ids.dtype)
    layer.step(*args)
    assert len(calls) == 2
    assert torch.equal(calls[0][0], layer.n1) and torch.equal(calls[1][0], layer.attn)
    for x, (a, b), before, after in calls:
        want, bound = lora_reference(x, a, b, layer.scales, ids, before, None)
        assert bool(((after.double() - want).abs() <= bound).all())
        assert torch.equal(after[ids < 0], before[ids < 0])
        # the bound is far below what the adapters add
        added = (want - before.double())[ids >= 0].norm(dim=1)
        assert bool((bound[ids >= 0].norm(dim=1) < 0.2 * added).all())
