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
