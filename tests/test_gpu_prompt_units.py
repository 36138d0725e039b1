"""Prompt attention where every CTA walks several units of several key tiles each, as ragged
prefill batches make it: what one unit leaves behind (places in the ring of copies, phases,
accumulators, flags of values that are not finite) is met by the next."""
import math

import pytest
import torch

import block_wise_fp8_gb300 as fb
from test_gpu_prompt_attention import BF16, I32, check, packed, reference, run

pytestmark = pytest.mark.gpu
RAGGED = [900, 33, 640, 1, 257, 511, 128, 400, 130]


def units(lens, HQ, HK):
    each = 2 * (128 // (HQ // HK))
    return sum(-(-n // each) for n in lens) * HK


@pytest.mark.parametrize("lens,HQ,HK,D", [
    (RAGGED, 32, 8, 128), (RAGGED, 24, 8, 64), (RAGGED, 32, 8, 80), (RAGGED, 64, 8, 16),
    ([400, 130, 257], 128, 1, 128), ([400, 130, 257], 100, 1, 64), ([1300] * 3, 24, 24, 128)])
def test_several_units_a_cta(lens, HQ, HK, D):
    assert units(lens, HQ, HK) > 2 * 152
    check(*run(lens, HQ, HK, D, seed=HQ + D, lead=3, tail=5))
    check(*run(lens, HQ, HK, D, seed=HQ + D + 1, spread=4.0))  # references that grow


@pytest.mark.parametrize("D", [64, 128])
def test_bad_values_in_some_units(D):
    """NaN and infinities in a few keys and values: the rows that see them, in their place;
    the other rows, and units that take over the others' buffers, are as without."""
    HQ, HK = 32, 8
    at = [5, 899, 930, 1200, 1573, 1700, 1832, 2400]  # rows, in five of the sequences
    bad = [math.nan, math.inf, -math.inf, math.nan, math.inf, -math.inf, math.inf, math.nan]

    def edit(q, k, v):
        for i, (row, x) in enumerate(zip(at, bad)):
            v[row, i % HK, (7 * i) % D] = x
        k[2700, 3, 1] = math.nan

    out, want, bound = run(RAGGED, HQ, HK, D, seed=D, edit=edit)
    hidden = torch.zeros_like(want, dtype=torch.bool)
    hidden[2700:2870, 12:16] = True  # the rows of the sequence behind the key that is NaN
    assert bool(out[hidden].isnan().all()) and bool(want[hidden].isnan().all())
    bad_place = ~want.isfinite()
    assert int(bad_place.sum()) > hidden.sum()
    assert bool((~out[bad_place].isfinite()).all())
    same = want.isinf()
    assert torch.equal(out[same], want[same])
    check(out[~bad_place], want[~bad_place], bound[~bad_place])


def test_in_place_graphs_and_two_streams():
    """y = q, captured and replayed with other bounds, and two calls at once on two streams
    with a workspace each."""
    HQ, HK, D = 32, 8, 128
    g = torch.Generator("cuda").manual_seed(2)
    T = sum(RAGGED)
    q, k, v = packed(g, T, HQ, HK, D)
    cuts = [[0]]
    for n in RAGGED:
        cuts[0].append(cuts[0][-1] + n)
    cuts += [[0, 10, 10, 1500, 1501, 1700, 2222, 2500, 2999, 3000], [0] * 9 + [T]]
    off = torch.tensor(cuts[0], dtype=I32, device="cuda")
    ws = fb.new_workspace(fb.OP_PROMPT_ATTENTION, T, HQ, D)
    x = torch.empty(T, HQ, D, dtype=BF16, device="cuda")
    x.copy_(q)
    fb.fp8bq_prompt_attention(x, k, v, off, x, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fb.fp8bq_prompt_attention(x, k, v, off, x, ws)
    wants = []
    for c in cuts:
        want, bound = reference(q, k, v, c, D ** -0.5)
        off.copy_(torch.tensor(c, dtype=I32))
        x.copy_(q)
        graph.replay()
        check(x.double(), want, bound)
        wants.append(x.clone())
    streams = [torch.cuda.Stream() for _ in range(2)]
    offs = [torch.tensor(c, dtype=I32, device="cuda") for c in cuts[:2]]
    ys = [torch.empty_like(x) for _ in range(2)]
    spaces = [fb.new_workspace(fb.OP_PROMPT_ATTENTION, T, HQ, D) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                fb.fp8bq_prompt_attention(q, k, v, offs[i], ys[i], spaces[i])
    torch.cuda.synchronize()
    assert torch.equal(ys[0], wants[0]) and torch.equal(ys[1], wants[1])
    assert all(fb.fp8bq_poll_status(s) == 0 for s in (ws, *spaces))


def test_long_prompt():
    check(*run([6100, 300], 4, 2, 128, seed=1))
    check(*run([5000], 2, 1, 64, seed=2))


def test_strides_past_31_bits():
    """Token strides whose products pass 2^31 elements: the rows of a packed call."""
    T, HQ, HK, D = 3, 4, 2, 64
    g = torch.Generator("cuda").manual_seed(3)
    q, k, v = packed(g, T, HQ, HK, D)
    off = torch.tensor([0, T], dtype=I32, device="cuda")
    ws = fb.new_workspace(fb.OP_PROMPT_ATTENTION, T, HQ, D)
    y = torch.empty(T, HQ, D, dtype=BF16, device="cuda")
    fb.fp8bq_prompt_attention(q, k, v, off, y, ws)
    stride, wide = 2 ** 30 + 64, (2 * HQ + 2 * HK) * D
    buf = torch.empty((T - 1) * stride + wide, dtype=BF16, device="cuda")
    assert (T - 1) * stride > 2 ** 31

    def view(head, H):
        return buf.as_strided((T, H, D), (stride, D, 1), head * D)

    q2, k2, v2, y2 = view(0, HQ), view(HQ, HK), view(HQ + HK, HK), view(HQ + 2 * HK, HQ)
    q2.copy_(q), k2.copy_(k), v2.copy_(v)
    fb.fp8bq_prompt_attention(q2, k2, v2, off, y2, ws)
    assert torch.equal(y2, y)
