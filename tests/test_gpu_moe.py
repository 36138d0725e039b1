"""The whole MoE layer against its definition in 64 bits.

Bound of an output, from the formulas: half a BF16 step of the result (2^-8);
the binary32 sums of both products, (K + 64) * 2^-23 of their sums of
magnitudes (a step a term: the tensor core may truncate); and the hidden rows'
quantisation: what the first product's error moves h by can move an E4M3 code
whose quotient lies that near a rounding border, by one step.  Which codes those
are is computed here, element by element; every other code must be the same.
On top of it the relative Frobenius error of the GEMM tests (4e-3)."""
import json
import os
import subprocess
import sys

import pytest
import torch

import block_wise_fp8_gb300 as fb
from gpu_util import FROB_TOL, Guarded

pytestmark = pytest.mark.gpu
BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def experts(g, E, rows, cols):
    q = (torch.randn(E, rows, cols, generator=g, device="cuda") * 112).clamp(-448, 448)
    s = torch.rand(E, -(-rows // 128), -(-cols // 128), generator=g, device="cuda")
    return q.to(torch.float8_e4m3fn), (s + 0.5) * 2e-4


def inputs(M, E, H, I, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    w13, s13 = experts(g, E, 2 * I, H)
    w2, s2 = experts(g, E, H, I)
    x = torch.randn(M, H, generator=g, device="cuda").to(BF16)
    logits = torch.randn(M, E, generator=g, device="cuda") * 2
    return dict(x=x, logits=logits, w13=w13, s13=s13, w2=w2, s2=s2), g


def route_ref(l, topk, sigmoid, renorm, scale, bias=None):
    l = l.double()
    usable = ~(torch.isnan(l) | (l == float("-inf")))
    lc = torch.where(usable, l, float("-inf")).clamp(max=3.4028234663852886e38)
    if sigmoid:
        p = 1 / (1 + torch.exp(-lc))
    else:
        p = torch.exp(lc - lc.max(1, keepdim=True).values)
        p = p / p.sum(1, keepdim=True)
    key = lc if bias is None else torch.where(usable, p + bias.double(), float("-inf"))
    order = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :topk]
    got = usable.gather(1, order)
    w = torch.where(got, p.gather(1, order), 0.0)
    if renorm:
        s = w.sum(1, keepdim=True)
        w = torch.where(s > 0, w / s, 0.0)
    return torch.where(got, order, -1), w * scale


def e4m3_round(v):
    """(nearest E4M3 value, step there, distance to the nearest rounding border)"""
    e = (torch.frexp(v)[1].double() - 1).clamp(min=-6, max=8)
    step = torch.exp2(e - 3)
    r = v / step
    q = torch.round(r) * step
    return q, step, ((r - torch.floor(r)) - 0.5).abs() * step


def deq(q, s):
    rows, cols = q.shape
    i, j = torch.arange(rows, device="cuda") // 128, torch.arange(cols, device="cuda") // 128
    return q.double() * s.double()[i][:, j]


def quant_x(x):
    M, H = x.shape
    out = torch.zeros(M, H, dtype=torch.float64, device="cuda")
    for k in range(0, H, 128):
        b = x[:, k:k + 128].float()
        s = b.abs().amax(1, keepdim=True).clamp(min=1e-10) * torch.full((), 1 / 448, device="cuda")
        out[:, k:k + 128] = e4m3_round((b / s).double())[0].clamp(-448, 448) * s.double()
    return out


def reference(d, ids, w):
    x = quant_x(d["x"])
    M, H = x.shape
    I = d["w13"].shape[1] // 2
    y = torch.zeros(M, H, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(y)
    for e in range(d["w13"].shape[0]):
        tok, k = (ids == e).nonzero(as_tuple=True)
        if not tok.numel():
            continue
        W, W2 = deq(d["w13"][e], d["s13"][e]), deq(d["w2"][e], d["s2"][e])
        gu, mag = x[tok] @ W.t(), x[tok].abs() @ W.abs().t() * (H + 64) * 2.0 ** -23
        gate, up, dg, du = gu[:, :I], gu[:, I:], mag[:, :I], mag[:, I:]
        sg = 1 / (1 + torch.exp(-gate))
        h = gate * sg * up
        # |d(silu)/dg| <= 1.1, silu <= |g|; exp, division and product in binary32
        dh = 1.1 * dg * up.abs() + (gate * sg).abs() * du + dg * du + h.abs() * 2.0 ** -20
        hq, dq = torch.zeros_like(h), torch.zeros_like(h)
        for b in range(0, I, 128):
            hb, db = h[:, b:b + 128], dh[:, b:b + 128]
            amax, at = hb.abs().max(1, keepdim=True)
            s = amax.clamp(min=1e-10) / 448
            ds = (db.max(1, keepdim=True).values + amax * 2.0 ** -23) / 448  # scale's error
            q, step, border = e4m3_round(hb / s)
            dr = db / s + (hb / s).abs() * ds / s  # error of the quotient
            flip = torch.where(dr >= border, step * torch.ceil(dr / step + 0.5), 0.0)
            hq[:, b:b + 128] = q * s
            dq[:, b:b + 128] = flip * s + (q.abs() + flip) * ds
        o = hq @ W2.t()
        do = dq @ W2.abs().t() + hq.abs() @ W2.abs().t() * (I + 64) * 2.0 ** -23
        wk = w[tok, k].double()[:, None]
        y.index_add_(0, tok, o * wk)
        tol.index_add_(0, tok, (do + o.abs() * 2.0 ** -20) * wk.abs())
    return y, tol + (y.abs() + tol) * 2.0 ** -8


def check(y, ref, tol, frob=True):
    err = (y.double() - ref).abs()
    assert bool((err <= tol + 1e-30).all()), float((err / tol.clamp(min=1e-30)).max())
    if frob and float(ref.norm()) > 0:
        assert float(err.norm() / ref.norm()) <= FROB_TOL


def run(d, topk, ws=None, **kw):
    M, H = d["x"].shape
    E, I2, _ = d["w13"].shape
    ws = fb.new_moe_workspace(M, E, H, I2 // 2, topk) if ws is None else ws
    y = torch.full((M, H), 9.0, device="cuda", dtype=BF16)
    ids = torch.full((M, topk), -9, device="cuda", dtype=I32)
    w = torch.full((M, topk), -9.0, device="cuda", dtype=F32)
    fb.fp8bq_moe_layer(d["x"], d["logits"], d["w13"], d["s13"], d["w2"], d["s2"], y, ws, topk,
                       ids_out=ids, weights_out=w, **kw)
    assert fb.fp8bq_poll_status(ws) == 0
    return y, ids, w


def check_all(d, topk, got, sigmoid, renorm, scale, bias=None, frob=True):
    y, ids, w = got
    rid, rw = route_ref(d["logits"], topk, sigmoid, renorm, scale, bias)
    assert torch.equal(ids.long(), rid)
    # exp, sum and quotients in binary32: E + 32 roundings at most
    assert bool(((w.double() - rw).abs() <= rw.abs() * (d["logits"].shape[1] + 32) * 2.0 ** -24
                 + 1e-37).all())
    check(y, *reference(d, rid, rw), frob=frob)


@pytest.mark.parametrize("M,E,H,I,topk", [
    (1, 1, 16, 128, 1), (1, 8, 128, 128, 2), (2, 3, 144, 128, 3), (3, 4, 272, 256, 4),
    (1, 64, 2048, 768, 4), (16, 8, 512, 384, 3), (17, 8, 528, 256, 8), (33, 64, 1040, 128, 6),
    (64, 4, 256, 128, 2), (61, 2, 400, 256, 2), (64, 512, 256, 128, 16), (40, 33, 384, 128, 1),
    (5, 16, 1168, 640, 10)])
def test_layer(M, E, H, I, topk):
    d, g = inputs(M, E, H, I, seed=M * 100 + E)
    for score, renorm, scale in ((fb.MOE_SOFTMAX, True, 1.0), (fb.MOE_SIGMOID, False, 2.5)):
        got = run(d, topk, score=score, renormalize=renorm, routed_scale=scale)
        check_all(d, topk, got, score == fb.MOE_SIGMOID, renorm, scale)


def test_one_workspace_serves_changing_routes_and_repeats_are_identical():
    d, g = inputs(24, 16, 512, 256, seed=1)
    ws = fb.new_moe_workspace(24, 16, 512, 256, 4)
    for i in range(6):
        d["logits"] = torch.randn(24, 16, generator=g, device="cuda") * (10 if i % 2 else 1)
        got = run(d, 4, ws=ws)
        check_all(d, 4, got, False, True, 1.0)
        assert torch.equal(got[0], run(d, 4, ws=ws)[0])


def test_one_workspace_serves_calls_of_several_sizes():
    sizes = [(64, 40, 256, 256, 16), (1, 3, 1040, 512, 2), (20, 64, 128, 128, 5), (64, 8, 512, 128, 8),
             (1, 1, 16, 128, 1), (33, 40, 256, 384, 16)]
    ws = torch.empty(max(fb.fp8bq_moe_workspace_bytes(*v) for v in sizes), dtype=U8, device="cuda")
    ws.zero_()
    for i, (M, E, H, I, topk) in enumerate(sizes + sizes[::-1]):
        d, _ = inputs(M, E, H, I, seed=60 + i)
        check_all(d, topk, run(d, topk, ws=ws), False, True, 1.0)


def test_choice_by_bias_and_close_scores():
    d, g = inputs(32, 96, 256, 128, seed=2)
    bias = torch.randn(96, generator=g, device="cuda") * 0.3
    got = run(d, 6, score=fb.MOE_SIGMOID, bias=bias)
    check_all(d, 6, got, True, True, 1.0, bias)
    # scores that binary32 cannot tell apart: logits near 16, where the sigmoid
    # is 1 - 1e-7, with one bias for all
    d["logits"] = 16 + torch.rand(32, 96, generator=g, device="cuda")
    bias = torch.full((96,), 0.7, device="cuda")
    got = run(d, 6, score=fb.MOE_SIGMOID, bias=bias)
    check_all(d, 6, got, True, True, 1.0, bias)


def test_ties_go_to_the_lower_index():
    d, _ = inputs(4, 40, 128, 128, seed=3)
    d["logits"].zero_()
    d["logits"][1, 35] = d["logits"][1, 7] = 1.0
    got = run(d, 3)
    assert got[1].tolist() == [[0, 1, 2], [7, 35, 0], [0, 1, 2], [0, 1, 2]]
    check_all(d, 3, got, False, True, 1.0)


@pytest.mark.parametrize("score", [0, 1])
def test_masked_logits(score):
    d, _ = inputs(5, 12, 256, 128, seed=4)
    inf, nan = float("inf"), float("nan")
    d["logits"][0] = -inf                      # nothing left
    d["logits"][1, 1:] = -inf                  # one expert left
    d["logits"][2] = nan
    d["logits"][2, 3] = 0.5                    # one number among NaN
    d["logits"][3, 2] = d["logits"][3, 9] = inf
    d["logits"][4] = -3.402823466e38           # the lowest value is a value
    got = run(d, 4, score=score, renormalize=True)
    assert got[1][0].tolist() == [-1] * 4 and bool((got[0][0] == 0).all())
    assert got[1][1].tolist() == [0, -1, -1, -1] and got[1][2].tolist() == [3, -1, -1, -1]
    assert got[1][3, :2].tolist() == [2, 9] and got[1][4].tolist() == [0, 1, 2, 3]
    check_all(d, 4, got, score == 1, True, 1.0)


def test_every_token_masked():
    d, _ = inputs(3, 4, 400, 128, seed=5)
    d["logits"].fill_(float("-inf"))
    y, ids, w = run(d, 2)
    assert bool((y == 0).all() and (ids == -1).all() and (w == 0).all())


@pytest.mark.parametrize("M,E,H,I,topk", [(1, 8, 256, 128, 4), (20, 6, 400, 256, 5),
                                          (64, 3, 128, 128, 3)])
def test_tokens_routed_by_the_caller(M, E, H, I, topk):
    d, g = inputs(M, E, H, I, seed=6)
    ids = torch.randint(-2, E + 2, (M, topk), generator=g, device="cuda", dtype=I32)
    w = torch.randn(M, topk, generator=g, device="cuda")
    y = torch.full((M, H), 9.0, device="cuda", dtype=BF16)
    ws = fb.new_moe_workspace(M, E, H, I, topk)
    fb.fp8bq_moe_experts(d["x"], ids, w, d["w13"], d["s13"], d["w2"], d["s2"], y, ws)
    assert fb.fp8bq_poll_status(ws) == 0
    check(y, *reference(d, ids.long(), w))


@pytest.mark.parametrize("M", [3, 40])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_nonfinite_inputs_stay_in_their_token(M, value):
    d, _ = inputs(M, 6, 272, 256, seed=70)
    clean = run(d, 2)
    d["x"][1, 200] = value
    got = run(d, 2)
    assert bool(got[0][1].isnan().all())       # the group's scale or its code is no number
    rest = torch.arange(M, device="cuda") != 1
    assert torch.equal(got[0][rest], clean[0][rest])
    assert torch.equal(got[1], clean[1]) and torch.equal(got[2], clean[2])


def test_zero_rows_pitched_input_and_guarded_output():
    M, E, H, I, topk = 6, 5, 272, 128, 2
    d, _ = inputs(M, E, H, I, seed=7)
    d["x"][2] = 0
    wide = torch.full((M, H + 40), float("nan"), device="cuda", dtype=BF16)
    wide[:, :H] = d["x"]
    d["x"] = wide[:, :H]
    out = Guarded((M, H), BF16, fill=9.0)
    ws = Guarded((fb.fp8bq_moe_workspace_bytes(M, E, H, I, topk),), U8)
    fb.fp8bq_workspace_init(ws.t)
    fb.fp8bq_moe_layer(d["x"], d["logits"], d["w13"], d["s13"], d["w2"], d["s2"], out.t, ws.t, topk)
    assert fb.fp8bq_poll_status(ws.t) == 0
    out.check("y")
    ws.check("ws")
    rid, rw = route_ref(d["logits"], topk, False, True, 1.0)
    check(out.t, *reference(d, rid, rw))
    assert bool((out.t[2] == 0).all())


def test_capture_replays_with_new_inputs():
    d, g = inputs(9, 16, 512, 256, seed=8)
    ws = fb.new_moe_workspace(9, 16, 512, 256, 4)
    y = torch.empty(9, 512, device="cuda", dtype=BF16)

    def call():
        fb.fp8bq_moe_layer(d["x"], d["logits"], d["w13"], d["s13"], d["w2"], d["s2"], y, ws, 4)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        d["x"].copy_(torch.randn(9, 512, generator=g, device="cuda"))
        d["logits"].copy_(torch.randn(9, 16, generator=g, device="cuda"))
        graph.replay()
        rid, rw = route_ref(d["logits"], 4, False, True, 1.0)
        check(y, *reference(d, rid, rw))
    assert fb.fp8bq_poll_status(ws) == 0


def test_agrees_with_the_grouped_gemms():
    """The layer's first product is the grouped GEMM's: one expert, weights of one."""
    M, H, I = 16, 1024, 256
    d, _ = inputs(M, 1, H, I, seed=9)
    y = torch.empty(M, H, device="cuda", dtype=BF16)
    ws = fb.new_moe_workspace(M, 1, H, I, 1)
    ids, w = torch.zeros(M, 1, device="cuda", dtype=I32), torch.ones(M, 1, device="cuda")
    fb.fp8bq_moe_experts(d["x"], ids, w, d["w13"], d["s13"], d["w2"], d["s2"], y, ws)
    off = torch.tensor([0, M], device="cuda", dtype=I32)

    def grouped(x, wt, sc):
        K, N = x.shape[1], wt.shape[1]
        q, s = torch.empty(M, K, device="cuda", dtype=U8), torch.empty(M, -(-K // 128), device="cuda")
        fb.fp8bq_quant_act(x, q, s)
        o = torch.empty(M, N, device="cuda", dtype=BF16)
        fb.fp8bq_grouped_gemm(q, s, wt, sc, off, o, fb.new_workspace(fb.OP_GROUPED_GEMM, M, N, K))
        return o
    gu = grouped(d["x"], d["w13"], d["s13"]).float()
    h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
    o = grouped(h.to(BF16), d["w2"], d["s2"]).float()
    # that path rounds g, u and h to BF16, which moves E4M3 codes: 2^-4 of single
    # values, averaged over I of them
    assert float((y.float() - o).norm() / o.norm()) < 2.0 ** -5


CHILD = r"""
import json, torch
import block_wise_fp8_gb300 as fb
from test_gpu_moe import inputs, run, check_all
res = []
for M in (1, 40):
    d, _ = inputs(M, 8, 512, 256, seed=M)
    ws = fb.new_moe_workspace(M, 8, 512, 256, 2)
    y = torch.empty(M, 512, device="cuda", dtype=torch.bfloat16)
    fb.fp8bq_moe_layer(d["x"], d["logits"], d["w13"], d["s13"], d["w2"], d["s2"], y, ws, 2)
    res.append(fb.fp8bq_poll_status(ws))
for M in (1, 40):
    d, _ = inputs(M, 8, 512, 256, seed=M)
    check_all(d, 2, run(d, 2), False, True, 1.0)
print("RESULT " + json.dumps(res))
"""


def test_a_wait_that_runs_out_is_reported():
    """CTA 0 skips its first weight tile: every wait behind it is bounded, the
    status says so, and the next calls on fresh workspaces are right."""
    env = dict(os.environ, FP8BQ_FAULT_INJECT="skip_first_load:2", FP8BQ_WAIT_LIMIT_MS="50",
               PYTHONPATH=ROOT + os.pathsep + os.path.join(ROOT, "tests"))
    p = subprocess.run([sys.executable, "-c", CHILD], env=env, cwd=ROOT, capture_output=True,
                       text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-2000:]
    line = [v for v in p.stdout.splitlines() if v.startswith("RESULT ")][0]
    assert json.loads(line[7:]) == [8, 8]


@pytest.mark.parametrize("mask", [torch.finfo(F32).min, -1e30, float("-inf")])
@pytest.mark.parametrize("E", [33, 96, 130, 500])
def test_experts_masked_by_their_bias(E, mask):
    """Fewer experts are free than are chosen: the masked ones follow by their
    index, each once, or, at -inf, not at all; a masked logit never does."""
    M, topk = 9, 6
    d, g = inputs(M, E, 256, 128, seed=E)
    bias = torch.full((E,), mask, device="cuda")
    free = [E - 1, 7, E // 2]
    bias[free] = torch.tensor([0.3, 0.1, 0.2], device="cuda")
    d["logits"][:, 2] = float("-inf")
    d["logits"][3, 7] = float("nan")
    got = run(d, topk, score=fb.MOE_SIGMOID, bias=bias)
    usable = d["logits"] > float("-inf")
    key = torch.where(usable, torch.sigmoid(d["logits"].double()) + bias.double(), float("-inf"))
    order = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :topk]
    rid = torch.where(key.gather(1, order) > float("-inf"), order, -1)
    assert torch.equal(got[1].long(), rid)
    w = torch.where(rid >= 0, torch.sigmoid(d["logits"].double()).gather(1, rid.clamp(min=0)), 0.0)
    w = w / w.sum(1, keepdim=True)
    # exp, sum and quotient in binary32, as in check_all
    assert bool(((got[2].double() - w).abs() <= w * (E + 32) * 2.0 ** -24 + 1e-37).all())
    check(got[0], *reference(d, rid, w))


@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("top", [-20.0, -87.0, -90.0, -200.0, -700.0])
def test_renormalised_weights_of_very_negative_logits(top, with_bias):
    """Sigmoids that are small or nothing in binary32 still have shares."""
    M, E, topk = 5, 12, 4
    d, g = inputs(M, E, 256, 128, seed=11)
    d["logits"] = top - 3 * torch.rand(M, E, generator=g, device="cuda")
    d["logits"][1] = top                       # equal shares
    d["logits"][2, 4:] -= 60                   # shares of very different size
    d["logits"][3, ::2] = float("-inf")
    d["logits"][4, 1:] -= 300                  # one share is all there is
    bias = torch.randn(E, generator=g, device="cuda") if with_bias else None
    got = run(d, topk, score=fb.MOE_SIGMOID, renormalize=True, routed_scale=2.5, bias=bias)
    check_all(d, topk, got, True, True, 2.5, bias)
    assert bool(((got[2].sum(1) - 2.5).abs() < 1e-5).all())
