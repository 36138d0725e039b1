"""The decoder layer example with the library's attention: prompts, then tokens over the
4-bit cache, then what is left of it after an eviction.

The attention's own rounding is far below that of the E4M3 activations before the four
products (test_gpu_layer_example.py has their bounds), and the 64-bit form reads the keys
and values that the cache holds, so the same bounds serve: the residual within 2^-4, the
experts' output within 2^-2."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

import block_wise_fp8_gb300 as fb  # noqa: E402
import decoder_layer  # noqa: E402

SIZES = dict(H=1024, heads=8, kv_heads=2, D=128, E=16, I=256, topk=4, adapters=4, rank=24)


def agree(layer, args, **kw):
    y, r = layer.step(*args, **kw)
    for ws in (layer.ws_moe, layer.ws_lora, layer.ws_o, layer.ws_qkv, layer.ws_prompt):
        assert fb.fp8bq_poll_status(ws) == 0
    ry, rr = layer.reference(*args, **kw)
    assert float((r.double() - rr).norm() / rr.norm()) < 2.0 ** -4
    assert float((y.double() - ry).norm() / ry.norm()) < 2.0 ** -2


@pytest.mark.parametrize("bounds", [[0, 1], [0, 5, 6, 33], [0, 64], [0, 20, 40, 57]])
def test_prompts(bounds):
    layer = decoder_layer.Layer(bounds[-1], context=1, **SIZES)
    args = decoder_layer.inputs(layer, seed=len(bounds), adapters=4)
    agree(layer, args, offsets=torch.tensor(bounds, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("M", [1, 5, 33])
def test_tokens_over_the_cache_and_eviction(M):
    layer = decoder_layer.Layer(M, context=45, cache4=True, page=16, **SIZES)
    for n in range(3):
        before = layer.weights.double().sum()
        agree(layer, decoder_layer.inputs(layer, seed=n, adapters=4))
        # every query row hands out a weight of one
        assert abs(float(layer.weights.double().sum() - before) - M * 8) < M * 8 * 2.0 ** -18
        layer.lens += 1
    assert fb.fp8bq_poll_status(layer.ws_kv4) == 0
    at = torch.arange(48, device="cuda").repeat(M, 1)
    who = torch.arange(M, device="cuda")[:, None]
    old_k, old_v = [t.view(M, 48, 2, 128) for t in layer.read_rows(layer.slots(who, at).flatten())]
    kept = layer.evict(20, 4).long()
    assert layer.lens.tolist() == [20] * M
    assert torch.equal(kept[:, :, -4:], torch.arange(44, 48, device="cuda").expand(M, 2, 4))
    new_k, new_v = [t.view(M, 20, 2, 128)
                    for t in layer.read_rows(layer.slots(who, at[:, :20]).flatten())]
    for h in range(2):
        pick = kept[:, h, :, None].expand(-1, -1, 128)
        assert torch.equal(new_k[:, :, h], old_k[:, :, h].gather(1, pick))
        assert torch.equal(new_v[:, :, h], old_v[:, :, h].gather(1, pick))
    agree(layer, decoder_layer.inputs(layer, seed=7, adapters=4))


def test_prompt_rows_into_the_cache():
    """A prompt's rows, written to the cache, are what its next token attends to."""
    M, D = 24, 128
    layer = decoder_layer.Layer(M, context=1, **SIZES)
    args = decoder_layer.inputs(layer, seed=3, adapters=4)
    layer.step(*args, offsets=torch.tensor([0, M], dtype=torch.int32, device="cuda"))
    nq, nk = layer.heads * D, layer.kv * D
    v = layer.qkv[:, nq + nk:].view(M, layer.kv, D)
    cache = fb.new_kv4_cache(3, layer.kv, 16, D)
    table = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    at = torch.arange(M, device="cuda")
    slots = table[0].long()[at // 16] * 16 + at % 16
    fb.fp8bq_kv4_append(layer.k, v, slots, cache)
    ws = fb.new_kv4_workspace(1, 1, layer.heads, layer.kv, D, 32)
    y = torch.empty(1, layer.heads, D, dtype=torch.bfloat16, device="cuda")
    fb.fp8bq_kv4_attention(layer.q[-1:], cache, table,
                           torch.tensor([M], dtype=torch.int32, device="cuda"), y, ws)
    # the prompt's last row saw the same keys and values before their rounding to four
    # bits: E2M1 is off by a quarter of a value at most (half a step of 2^-1), the scale
    # of 16 values by 2^-4; a mean over 24 such rows stays well within their size
    want = layer.attn[-1].view(layer.heads, D).double()
    assert float((y[0].double() - want).norm() / want.norm()) < 0.5
    k4, v4 = torch.empty_like(layer.k), torch.empty_like(layer.k)
    fb.fp8bq_kv4_read(cache, slots, k4, v4)
    g = layer.heads // layer.kv
    s = torch.einsum("hd,jhd->hj", layer.q[-1].double(), k4.double().repeat_interleave(g, 1)) * D ** -0.5
    p = torch.softmax(s, -1)
    exact = torch.einsum("hj,jhd->hd", p, v4.double().repeat_interleave(g, 1))
    size = torch.einsum("hj,jhd->hd", p, v4.double().abs().repeat_interleave(g, 1))
    # half a step of BF16 for the output, of FP16 for the weights, and FP32 sums
    assert bool(((y[0].double() - exact).abs() <= exact.abs() * 2.0 ** -8 + size * 2.0 ** -10).all())


def test_slots_behind_the_table():
    """A request without room: its token is left out, and the pages stay as they were."""
    layer = decoder_layer.Layer(3, context=45, cache4=True, page=16, **SIZES)
    room = layer.pages.shape[1] * 16
    layer.lens.copy_(torch.tensor([room, 45, room + 40]))
    got = layer.slots(torch.arange(3, device="cuda"), layer.lens.long())
    assert got[0] == got[2] == -1 and got[1] == int(layer.pages[1, 2]) * 16 + 13
    before = layer.cache4.clone()
    layer.step(*decoder_layer.inputs(layer, adapters=4))
    assert fb.fp8bq_poll_status(layer.ws_kv4) == 0
    changed = (layer.cache4 != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert changed == [int(layer.pages[1, 2])]
