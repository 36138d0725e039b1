"""Adapter grouping and the adapters' products against plain forms in 64 bits.

Bound of y: half a BF16 step of the result (2^-8), t = A x held with 16
significant bits (2^-17 of each term b t), and binary32 sums of K and of R + 1
terms: (K + R + 64) * 2^-23 of the sums of magnitudes (one step, not half, a
term: the tensor instruction may truncate)."""
import json
import os
import subprocess
import sys

import pytest
import torch

import block_wise_fp8_gb300 as fb

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def group_ref(ids, L):
    key = torch.where((ids >= 0) & (ids < L), ids, L).long().cpu()
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=L + 1)[:L]
    return order.to(I32), torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]).to(I32)


def group(ids, L):
    order = torch.full((ids.numel(),), -7, device="cuda", dtype=I32)
    offsets = torch.full((L + 1,), -7, device="cuda", dtype=I32)
    fb.fp8bq_lora_group(ids, order, offsets)
    return order, offsets


@pytest.mark.parametrize("M,L", [(0, 3), (1, 1), (31, 5), (32, 512), (33, 2), (1000, 7),
                                 (1025, 512), (16384, 128), (100003, 33),
                                 (1024, 9), (2048, 1), (2049, 40), (8191, 511), (8193, 300)])
def test_group_sorts_stably(M, L):
    g = torch.Generator("cuda").manual_seed(M + L)
    ids = torch.randint(-2, L + 2, (M,), generator=g, device="cuda", dtype=I32)
    order, offsets = group(ids, L)
    ro, rf = group_ref(ids, L)
    assert torch.equal(offsets.cpu(), rf)
    assert torch.equal(order.cpu(), ro)


@pytest.mark.parametrize("value", [0, 4, -1])
def test_group_of_one_key(value):
    ids = torch.full((777,), value, device="cuda", dtype=I32)
    order, offsets = group(ids, 5)
    ro, rf = group_ref(ids, 5)
    assert torch.equal(offsets.cpu(), rf) and torch.equal(order.cpu(), ro)


def reference(x, a, b, scales, ids, base, ranks):
    L, R, K = a.shape
    y = base.double().clone()
    tol = torch.zeros_like(y)
    for i in range(L):
        tok = (ids == i).nonzero(as_tuple=True)[0]
        r = R if ranks is None else int(ranks[i].clamp(0, R))
        if not tok.numel() or r == 0:
            continue
        xa, aa, ba, s = x[tok].double(), a[i, :r].double(), b[i, :, :r].double(), scales[i].double()
        t = xa @ aa.t()
        y[tok] += s * (t @ ba.t())
        tol[tok] = s.abs() * (t.abs() @ ba.abs().t() * 2.0 ** -17 +
                              xa.abs() @ aa.abs().t() @ ba.abs().t() * (K + R + 64) * 2.0 ** -23)
    return y, tol + (y.abs() + tol) * 2.0 ** -8 + base.double().abs() * 2.0 ** -22


def inputs(M, L, R, K, N, seed, low=-1):
    g = torch.Generator("cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return dict(x=rn(M, K).to(BF16), a=(rn(L, R, K) * K ** -0.5).to(BF16),
                b=rn(L, N, R).to(BF16), scales=rn(L), base=(2 * rn(M, N)).to(BF16),
                ids=torch.randint(low, L, (M,), generator=g, device="cuda", dtype=I32))


def run(d, ranks=None, y=None, base=None):
    M, K = d["x"].shape
    L, R, _ = d["a"].shape
    order, offsets = group(d["ids"], L)
    base = d["base"] if base is None else base
    y = torch.full(base.shape, 5.0, device="cuda", dtype=BF16) if y is None else y
    ws = fb.new_workspace(fb.OP_LORA_ADD, M, R, K)
    fb.fp8bq_lora_add(d["x"], d["a"], d["b"], d["scales"], order, offsets, base, y, ws, ranks=ranks)
    return y


def check(y, ref, bound):
    err = (y.double() - ref).abs()
    assert bool((err <= bound).all()), float((err / bound.clamp(min=1e-30)).max())


@pytest.mark.parametrize("M,L,R,K,N", [
    (1, 1, 8, 16, 8), (1, 4, 16, 6144, 6144), (2, 3, 24, 272, 40), (17, 2, 32, 1040, 136),
    (33, 1, 64, 528, 104), (64, 32, 16, 512, 1000), (129, 2, 40, 256, 264),
    (300, 3, 128, 400, 72), (517, 5, 72, 320, 328), (1500, 4, 64, 640, 512),
    (700, 200, 16, 128, 64), (256, 1, 8, 64, 8), (1000, 2, 120, 2064, 1160), (9000, 5, 48, 192, 400), (2500, 500, 16, 128, 72),
    (127, 1, 16, 256, 64), (128, 1, 16, 256, 64), (191, 4, 16, 256, 64), (192, 4, 16, 256, 64),
    # enough tokens and work for the form of many tokens
    (1400, 1, 128, 4112, 4104), (2600, 3, 72, 2064, 5000), (1700, 6, 48, 6000, 10008),
    (1300, 3, 120, 4096, 4360), (9000, 2, 24, 2064, 4104), (10300, 1, 16, 4112, 4104),
    (9000, 1, 8, 10256, 8200), (140, 1, 128, 192, 72712), (2000, 20, 64, 4096, 8192)])
def test_products(M, L, R, K, N):
    d = inputs(M, L, R, K, N, seed=M + R)
    y = run(d)
    check(y, *reference(d["x"], d["a"], d["b"], d["scales"], d["ids"], d["base"], None))


@pytest.mark.parametrize("M,K,N", [(5, 256, 128), (200, 256, 128), (900, 256, 128),
                                   (1900, 4096, 6800)])
def test_ranks_hide_what_lies_past_them(M, K, N):
    L, R = 6, 64
    d = inputs(M, L, R, K, N, seed=M, low=0)
    ranks = torch.tensor([0, 1, 7, 21, 64, 1000], device="cuda", dtype=I32)
    for i in range(L):
        r = min(int(ranks[i]), R)
        d["a"][i, r:] = float("nan")
        d["b"][i, :, r:] = float("inf")
    y = run(d, ranks=ranks)
    check(y, *reference(d["x"], d["a"], d["b"], d["scales"], d["ids"], d["base"], ranks))
    assert torch.equal(y[d["ids"] == 0], d["base"][d["ids"] == 0])


@pytest.mark.parametrize("M,R,K,N", [(5, 16, 256, 128), (200, 16, 256, 128), (900, 16, 256, 128),
                                     (1900, 64, 4096, 6800)])
def test_an_infinite_input_stays_infinite_and_in_its_row(M, R, K, N):
    L = 2
    d = inputs(M, L, R, K, N, seed=M, low=0)
    d["a"][:, :, 7] = 0.5
    d["b"][:, ::2, :] = d["b"][:, ::2, :].abs() + 0.25   # same signs: every term is +inf
    d["scales"].fill_(1.5)
    clean = run(d)
    d["x"][3, 7] = float("inf")
    y = run(d)
    assert bool((y[3, ::2] == float("inf")).all())
    ref, _ = reference(d["x"], d["a"], d["b"], d["scales"], d["ids"], d["base"], None)
    assert torch.equal(y[3].isnan(), ref[3].isnan())
    rest = torch.arange(M, device="cuda") != 3
    assert torch.equal(y[rest], clean[rest])


@pytest.mark.parametrize("M,R,K,N", [(3, 16, 144, 80), (190, 16, 144, 80), (530, 16, 144, 80),
                                     (1500, 64, 2064, 12008)])
def test_in_place_and_pitched(M, R, K, N):
    L = 3
    d = inputs(M, L, R, K, N, seed=9)
    d["x"] = torch.cat([d["x"], torch.full((M, 24), float("nan"), device="cuda", dtype=BF16)], 1)[:, :K]
    wide = torch.cat([d["base"], torch.full((M, 16), 3.0, device="cuda", dtype=BF16)], 1)
    view = wide[:, :N]
    ref = reference(d["x"], d["a"], d["b"], d["scales"], d["ids"], d["base"], None)
    run(d, y=view, base=view)
    check(view, *ref)
    assert bool((wide[:, N:] == 3.0).all())


@pytest.mark.parametrize("M,R,N", [(70, 16, 96), (700, 16, 96), (2000, 64, 12000)])
def test_no_token_has_an_adapter(M, R, N):
    d = inputs(M, 4, R, 128, N, seed=1)
    d["ids"].fill_(-1)
    assert torch.equal(run(d), d["base"])
    keep = d["base"].clone()
    assert torch.equal(run(d, y=keep, base=keep), d["base"])


@pytest.mark.parametrize("M,R,N", [(40, 16, 64), (400, 16, 64), (1600, 64, 13000)])
def test_bounds_and_indices_outside_the_tokens_touch_nothing(M, R, N):
    d = inputs(M, 2, R, 128, N, seed=2, low=0)
    order = torch.arange(M, device="cuda", dtype=I32)
    order[3], order[5] = -4, 4000
    offsets = torch.tensor([-9, 20, M + 500], device="cuda", dtype=I32)
    ids = torch.where(torch.arange(M, device="cuda") < 20, 0, 1).to(I32)
    ref, bound = reference(d["x"], d["a"], d["b"], d["scales"], ids, d["base"], None)
    y = torch.full_like(d["base"], 5.0)
    ws = fb.new_workspace(fb.OP_LORA_ADD, M, R, 128)
    fb.fp8bq_lora_add(d["x"], d["a"], d["b"], d["scales"], order, offsets, d["base"], y, ws)
    left = torch.ones(M, dtype=torch.bool, device="cuda")
    left[[3, 5]] = False
    check(y[left], ref[left], bound[left])
    assert bool((y[~left] == 5.0).all())


@pytest.mark.parametrize("M,R,N", [(130, 32, 256), (1100, 32, 256), (1800, 64, 11000)])
def test_repeats_are_identical_and_capture_replays(M, R, N):
    d = inputs(M, 3, R, 512, N, seed=5)
    first = run(d)
    assert torch.equal(first, run(d))
    order, offsets = group(d["ids"], 3)
    ws = fb.new_workspace(fb.OP_LORA_ADD, M, R, 512)
    y = torch.empty_like(first)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fb.fp8bq_lora_group(d["ids"], order, offsets)
        fb.fp8bq_lora_add(d["x"], d["a"], d["b"], d["scales"], order, offsets, d["base"], y, ws)
    d["ids"].copy_((d["ids"] + 2) % 3)
    graph.replay()
    check(y, *reference(d["x"], d["a"], d["b"], d["scales"], d["ids"], d["base"], None))


def test_one_workspace_serves_calls_of_several_shapes():
    shapes = [(600, 3, 64, 1024, 264), (5, 2, 128, 6144, 64), (2000, 40, 16, 256, 136),
              (260, 200, 72, 640, 48), (64, 7, 24, 512, 96), (1500, 3, 64, 6144, 8200)]
    ws = torch.zeros(max(fb.fp8bq_workspace_bytes(fb.OP_LORA_ADD, M, R, K)
                         for M, _, R, K, _ in shapes), dtype=torch.uint8, device="cuda")
    for i, (M, L, R, K, N) in enumerate(shapes + shapes[::-1]):
        d = inputs(M, L, R, K, N, seed=40 + i)
        order, offsets = group(d["ids"], L)
        y = torch.empty_like(d["base"])
        fb.fp8bq_lora_add(d["x"], d["a"], d["b"], d["scales"], order, offsets, d["base"], y, ws)
        check(y, *reference(d["x"], d["a"], d["b"], d["scales"], d["ids"], d["base"], None))
    assert fb.fp8bq_poll_status(ws) == 0


def test_a_stream_of_its_own():
    d = inputs(50, 2, 16, 256, 128, seed=6)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        y = run(d)
    st.synchronize()
    check(y, *reference(d["x"], d["a"], d["b"], d["scales"], d["ids"], d["base"], None))


def test_no_tokens():
    d = inputs(1, 2, 16, 64, 64, seed=7)
    e = torch.empty(0, 64, device="cuda", dtype=BF16)
    none = torch.empty(0, device="cuda", dtype=I32)
    fb.fp8bq_lora_add(e, d["a"], d["b"], d["scales"], none, torch.zeros(3, device="cuda", dtype=I32),
                      e, e, fb.new_workspace(fb.OP_LORA_ADD, 0, 16, 64))


@pytest.mark.parametrize("N", [40, 72, 128, 200, 1160])
def test_neighbouring_tokens_go_as_boxes(N):
    """Requests of many tokens in order: whole warps of neighbours, their ends,
    and rows in between that are left alone (pitched y, in place too)."""
    M, L, R, K = 1900, 3, 64, 10800  # enough work for the form of many tokens
    d = inputs(M, L, R, K, N, seed=N)
    d["ids"] = (torch.arange(M, device="cuda") // 237 % (L + 1) - 1).to(I32)
    ref = reference(d["x"], d["a"], d["b"], d["scales"], d["ids"], d["base"], None)
    check(run(d), *ref)
    wide = torch.full((M, N + 24), 3.0, device="cuda", dtype=BF16)
    wide[:, :N] = d["base"]
    run(d, y=wide[:, :N], base=wide[:, :N])
    check(wide[:, :N], *ref)
    assert bool((wide[:, N:] == 3.0).all())


@pytest.mark.parametrize("M,L,R,N,free", [(2100, 3, 16, 9000, 0.5), (1300, 6, 72, 16392, 0.1),
                                          (5000, 2, 24, 4104, 0.95), (3000, 40, 32, 8200, 0.3),
                                          (2100, 3, 64, 9976, 0.5), (5000, 2, 40, 8200, 0.95),
                                          (3000, 9, 64, 8200, 0.3), (1300, 2, 128, 8200, 0.1)])
def test_many_blocks_are_shared_out(M, L, R, N, free):
    """Enough blocks that CTAs take some of them in turn, among them runs of rows
    without an adapter and of adapters of rank 0."""
    d = inputs(M, L, R, 64, N, seed=M)
    g = torch.Generator("cuda").manual_seed(1)
    d["ids"] = torch.where(torch.rand(M, generator=g, device="cuda") < free, -1, d["ids"]).to(I32)
    ranks = torch.tensor([R - 8 * (i % 3) if i != 1 else 0 for i in range(L)], device="cuda", dtype=I32)
    order, offsets = group(d["ids"], L)
    ws = fb.new_workspace(fb.OP_LORA_ADD, M, R, 64)
    ref = reference(d["x"], d["a"], d["b"], d["scales"], d["ids"], d["base"], ranks)
    for _ in range(2):
        y = torch.full_like(d["base"], 5.0)
        fb.fp8bq_lora_add(d["x"], d["a"], d["b"], d["scales"], order, offsets, d["base"], y, ws,
                          ranks=ranks)
        assert fb.fp8bq_poll_status(ws) == 0
        check(y, *ref)


CHILD = r"""
import json, torch
import block_wise_fp8_gb300 as fb
from test_gpu_lora import inputs, group, run, check, reference
d = inputs(1500, 2, 64, 6144, 8200, seed=1)
order, offsets = group(d["ids"], 2)
ws = fb.new_workspace(fb.OP_LORA_ADD, 1500, 64, 6144)
y = torch.empty_like(d["base"])
fb.fp8bq_lora_add(d["x"], d["a"], d["b"], d["scales"], order, offsets, d["base"], y, ws)
res = [fb.fp8bq_poll_status(ws)]
check(run(d), *reference(d["x"], d["a"], d["b"], d["scales"], d["ids"], d["base"], None))
print("RESULT " + json.dumps(res))
"""


def test_a_wait_that_runs_out_is_reported():
    """The first CTA never hands over its first stage: the waits behind it are
    bounded, the status says so, and the next call on a fresh workspace is right."""
    env = dict(os.environ, FP8BQ_FAULT_INJECT="skip_first_load:1", FP8BQ_WAIT_LIMIT_MS="50",
               PYTHONPATH=ROOT + os.pathsep + os.path.join(ROOT, "tests"))
    p = subprocess.run([sys.executable, "-c", CHILD], env=env, cwd=ROOT, capture_output=True,
                       text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-2000:]
    line = [v for v in p.stdout.splitlines() if v.startswith("RESULT ")][0]
    assert json.loads(line[7:]) == [8]


GROUP_CHILD = r"""
import torch
from test_gpu_lora import group, group_ref
M, sizes = {M}, {sizes}
for L in sizes:
    g = torch.Generator("cuda").manual_seed(L)
    ids = torch.randint(-2, L + 2, (M,), generator=g, device="cuda", dtype=torch.int32)
    order, offsets = group(ids, L)
    ro, rf = group_ref(ids, L)
    assert torch.equal(offsets.cpu(), rf) and torch.equal(order.cpu(), ro), L
"""


@pytest.mark.parametrize("M", [64, 1024, 1025, 2000])
def test_group_of_any_number_of_adapters(M):
    """The counters' shared memory passes the default limit between L = 349 and
    384; in a process of its own, where no call with more adapters came before."""
    code = GROUP_CHILD.format(M=M, sizes=[1, 348, 349, 350, 351, 365, 366, 367, 382, 383, 384, 512])
    env = dict(os.environ, PYTHONPATH=ROOT + os.pathsep + os.path.join(ROOT, "tests"))
    p = subprocess.run([sys.executable, "-c", code], env=env, cwd=ROOT, capture_output=True,
                       text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-2000:]
