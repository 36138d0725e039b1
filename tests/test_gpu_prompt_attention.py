"""Causal attention over packed prompts against the formula in 64 bits.

A row's bound: half a step of BF16 (2^-8) for the output, the same of every weight
(the weights enter the second product as BF16), the scores' FP32 sums of D products
((D + 8) steps of 2^-23 of the sum of magnitudes, times the scale), an exponential's
argument (2^-22 of it) and value (2^-21), and FP32 sums over n keys ((n / 8 + 64)
steps of 2^-22)."""
import math

import pytest
import torch

import block_wise_fp8_gb300 as fb
from gpu_util import Guarded

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32


def reference(q, k, v, bounds, scale):
    T, HQ, D = q.shape
    G = HQ // k.shape[1]
    y = torch.zeros(T, HQ, D, dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(y)
    for a, b in zip(bounds, bounds[1:]):
        n = b - a
        for h in range(HQ if n > 0 else 0):
            qq, kk, vv = (x.double() for x in (q[a:b, h], k[a:b, h // G], v[a:b, h // G]))
            hidden = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
            s = (qq @ kk.t() * scale).masked_fill(hidden, -math.inf)
            mag = (qq.abs() @ kk.abs().t() * scale).masked_fill(hidden, 0.0)
            p = torch.softmax(s, -1)
            fine = torch.where(vv.isfinite(), vv, 0.0)
            o, size = p @ fine, p @ fine.abs()
            for j, d in (~vv.isfinite()).nonzero().tolist():  # for the rows that see it
                o[j:, d] += p[j:, j] * vv[j, d]
            big = s.masked_fill(hidden, 0.0).abs().amax(-1)
            ds = mag.amax(-1) * (D + 8) * 2.0 ** -23 + big * 2.0 ** -22 + 2.0 ** -21
            rel = 2.0 ** -8 + 2 * ds + (n / 8 + 64) * 2.0 ** -22
            y[a:b, h] = o
            bound[a:b, h] = o.abs() * 2.0 ** -8 + size * rel[:, None] * 1.01
    return y, bound


def packed(g, T, HQ, HK, D, scale=1.0):
    qkv = (torch.randn(T, (HQ + 2 * HK) * D, generator=g, device="cuda") * scale).to(BF16)
    return (qkv[:, a * D:b * D].view(T, b - a, D) for a, b in ((0, HQ), (HQ, HQ + HK),
                                                              (HQ + HK, HQ + 2 * HK)))


def run(lens, HQ, HK, D, seed=0, scale=None, lead=0, tail=0, edit=None, spread=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    T = lead + sum(lens) + tail
    q, k, v = packed(g, T, HQ, HK, D, spread)
    bounds = [lead]
    for n in lens:
        bounds.append(bounds[-1] + n)
    if edit:
        edit(q, k, v)
    off = torch.tensor(bounds, dtype=I32, device="cuda")
    y = Guarded((T, HQ, D), BF16, fill=7.0)
    ws = fb.new_workspace(fb.OP_PROMPT_ATTENTION, T, HQ, D)
    fb.fp8bq_prompt_attention(q, k, v, off, y.t, ws, scale=scale)
    assert fb.fp8bq_poll_status(ws) == 0
    y.check("y")
    first = y.t.clone()
    fb.fp8bq_prompt_attention(q, k, v, off, y.t, ws, scale=scale)
    assert torch.equal(first.view(torch.int16), y.t.view(torch.int16))
    want, bound = reference(q, k, v, bounds, D ** -0.5 if scale is None else scale)
    live = torch.zeros(T, dtype=torch.bool, device="cuda")
    live[bounds[0]:bounds[-1]] = True
    assert bool((y.t[~live] == 7.0).all())  # rows of no sequence are left as they were
    return y.t.double()[live], want[live], bound[live]


def check(out, want, bound):
    err = (out - want).abs()
    assert bool((err <= bound).all()), f"{float((err / bound).max())} of the bound"


@pytest.mark.parametrize("D", [16, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("HQ,HK", [(1, 1), (8, 2), (3, 1)])
def test_sizes_and_heads(D, HQ, HK):
    check(*run([1, 5, 128, 129, 64, 300], HQ, HK, D, seed=D + HQ))


@pytest.mark.parametrize("HQ,HK", [(5, 5), (7, 1), (12, 2), (16, 1), (33, 1), (64, 2), (100, 1),
                                   (128, 1)])
def test_groups(HQ, HK):
    check(*run([70, 1, 200], HQ, HK, 64, seed=HQ))


@pytest.mark.parametrize("lens", [[1], [2], [127], [128], [255], [256], [257], [513], [1025],
                                  [0, 3, 0, 0, 400, 0], [1] * 400, [2047, 2], [4000]])
def test_lengths(lens):
    check(*run(lens, 4, 2, 128, seed=len(lens) + lens[0]))


def test_rows_of_no_sequence():
    check(*run([150, 0, 33], 8, 2, 128, lead=13, tail=77))


@pytest.mark.parametrize("scale,spread", [(2.0, 1.0), (1e-4, 1.0), (None, 6.0), (None, 0.01)])
def test_sharp_and_flat_rows(scale, spread):
    check(*run([700, 90], 8, 2, 128, scale=scale, spread=spread))


@pytest.mark.parametrize("lens", [[40, 60], [300, 200], [129, 500]])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_hidden_values_have_no_part(lens, bad):
    """Rows before a bad key or value, and rows of other sequences, are as without it;
    the rows that see a bad value have it in its place alone."""
    a = lens[0]
    T = sum(lens)
    for at in (a - 1, a, a // 2, T - 1):
        for which in ("k", "v"):
            def edit(q, k, v):
                (k if which == "k" else v)[at, 0, 3] = bad
            out, want, bound = run(lens, 4, 2, 64, edit=edit)
            end = a if at < a else T
            hit = torch.zeros(T, 4, 64, dtype=torch.bool, device="cuda")
            if which == "v":
                hit[at:end, :2, 3] = True
            else:
                hit[at:end, :2] = True
            assert bool(((out - want).abs() <= bound)[~hit].all())
            if which == "v":
                assert bool((~out[hit].isfinite()).all())
            elif bad != bad:
                assert bool(out[hit].isnan().all())


def test_bad_rows_past_the_sequences():
    def edit(q, k, v):
        for x in (q, k, v):
            x[:13] = math.nan
            x[13 + 183:] = math.nan
    check(*run([150, 0, 33], 8, 2, 128, lead=13, tail=77, edit=edit))


@pytest.mark.parametrize("size", [1e6, 1e12, 1e16])
def test_scores_of_any_size(size):
    """Scores so far apart that one key has all of a row's weight: its value, exactly."""
    g = torch.Generator("cuda").manual_seed(6)
    T, HQ, HK, D = 400, 4, 2, 128
    q, k, v = packed(g, T, HQ, HK, D)
    q.mul_(size), k.mul_(size)
    y = torch.empty(T, HQ, D, dtype=BF16, device="cuda")
    ws = fb.new_workspace(fb.OP_PROMPT_ATTENTION, T, HQ, D)
    fb.fp8bq_prompt_attention(q, k, v, torch.tensor([0, T], dtype=I32, device="cuda"), y, ws)
    s = torch.einsum("ihd,jhd->hij", q.double(), k.double().repeat_interleave(2, 1))
    s = s.masked_fill(torch.ones(T, T, dtype=torch.bool, device="cuda").triu(1), -math.inf)
    top = s.topk(2, -1)
    # FP32 sums cannot turn which of the two is larger, and e^-200 of the other is nothing
    mag = torch.einsum("ihd,jhd->hij", q.double().abs(), k.double().abs().repeat_interleave(2, 1))
    clear = (top.values[..., 0] - top.values[..., 1]) > mag.amax(-1) * (D + 8) * 2.0 ** -22 + 200 * D ** 0.5
    clear[:, 0] = True
    want = v.repeat_interleave(2, 1).transpose(0, 1).gather(1, top.indices[..., :1].expand(-1, -1, D))
    assert float(clear.float().mean()) > 0.9
    assert torch.equal(y.transpose(0, 1)[clear], want[clear])
    assert bool(y.isfinite().all())


def test_in_place_and_other_layouts():
    g = torch.Generator("cuda").manual_seed(3)
    T, HQ, HK, D = 333, 8, 2, 128
    q, k, v = packed(g, T, HQ, HK, D)
    off = torch.tensor([0, 100, T], dtype=I32, device="cuda")
    ws = fb.new_workspace(fb.OP_PROMPT_ATTENTION, T, HQ, D)
    y = torch.empty(T, HQ, D, dtype=BF16, device="cuda")
    fb.fp8bq_prompt_attention(q, k, v, off, y, ws)
    # heads outermost, padded rows
    qh = torch.empty(HQ, T, D + 8, dtype=BF16, device="cuda")[:, :, :D].transpose(0, 1)
    kh = torch.empty(HK, T, D, dtype=BF16, device="cuda").transpose(0, 1)
    vh = torch.empty(T + 5, HK + 1, D, dtype=BF16, device="cuda")[5:, 1:]
    qh.copy_(q), kh.copy_(k), vh.copy_(v)
    yh = torch.zeros(HQ, T, D + 24, dtype=BF16, device="cuda")
    fb.fp8bq_prompt_attention(qh, kh, vh, off, yh[:, :, 8:D + 8].transpose(0, 1), ws)
    assert torch.equal(yh[:, :, 8:D + 8].transpose(0, 1), y)
    assert bool((yh[:, :, :8] == 0).all()) and bool((yh[:, :, D + 8:] == 0).all())
    fb.fp8bq_prompt_attention(q, k, v, off, q, ws)
    assert torch.equal(q, y)


def test_streams_and_graphs():
    g = torch.Generator("cuda").manual_seed(9)
    T, HQ, HK, D = 600, 8, 2, 64
    q, k, v = packed(g, T, HQ, HK, D)
    off = torch.tensor([0, 100, 350, T], dtype=I32, device="cuda")
    y = torch.empty(T, HQ, D, dtype=BF16, device="cuda")
    ws = fb.new_workspace(fb.OP_PROMPT_ATTENTION, T, HQ, D)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        fb.fp8bq_prompt_attention(q, k, v, off, y, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fb.fp8bq_prompt_attention(q, k, v, off, y, ws)
    for cuts in ([0, 100, 350, T], [0, 1, 2, T], [0, 0, 599, T]):
        off.copy_(torch.tensor(cuts, dtype=I32))
        q.copy_(torch.randn(T, HQ, D, generator=g, device="cuda"))
        graph.replay()
        check(y.double(), *reference(q, k, v, cuts, D ** -0.5))


def test_bounds_outside_the_rows_are_clamped():
    g = torch.Generator("cuda").manual_seed(4)
    q, k, v = packed(g, 50, 4, 2, 64)
    y = torch.full((50, 4, 64), 7.0, dtype=BF16, device="cuda")
    ws = fb.new_workspace(fb.OP_PROMPT_ATTENTION, 50, 4, 64)
    fb.fp8bq_prompt_attention(q, k, v, torch.tensor([-9, 20, 10 ** 9], dtype=I32, device="cuda"), y, ws)
    check(y.double(), *reference(q, k, v, [0, 20, 50], 0.125))


def test_no_rows_at_all():
    """Sequences that are all empty, or none: nothing is written."""
    g = torch.Generator("cuda").manual_seed(5)
    q, k, v = packed(g, 50, 4, 2, 128)
    ws = fb.new_workspace(fb.OP_PROMPT_ATTENTION, 50, 4, 128)
    for cuts in ([0], [0, 0, 0], [50, 50], [70, 70, 90], [30, 10]):
        y = torch.full((50, 4, 128), 7.0, dtype=BF16, device="cuda")
        fb.fp8bq_prompt_attention(q, k, v, torch.tensor(cuts, dtype=I32, device="cuda"), y, ws)
        assert bool((y == 7.0).all()), cuts
    e = torch.empty(0, 4, 128, dtype=BF16, device="cuda")
    fb.fp8bq_prompt_attention(e, e[:, :2], e[:, :2], torch.zeros(2, dtype=I32, device="cuda"), e, ws)
    assert fb.fp8bq_poll_status(ws) == 0
