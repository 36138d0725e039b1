"""A copy that never lands, made on purpose in a child process as in test_gpu_fault.py: the
attention kernels' waits run out, they report it through the workspace's status word and
leave, and the next calls on zeroed workspaces are right."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import json
import torch
import block_wise_fp8_gb300 as fb
import test_gpu_kv4 as kv4
import test_gpu_prompt_attention as pa

res = {}

def prompt(D, lens, check=False):
    g = torch.Generator("cuda").manual_seed(1)
    q, k, v = pa.packed(g, sum(lens), 4, 2, D)
    bounds = [0]
    for n in lens:
        bounds.append(bounds[-1] + n)
    off = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    y = torch.empty(sum(lens), 4, D, dtype=torch.bfloat16, device="cuda")
    ws = fb.new_workspace(fb.OP_PROMPT_ATTENTION, sum(lens), 4, D)
    fb.fp8bq_prompt_attention(q, k, v, off, y, ws)
    st = fb.fp8bq_poll_status(ws)
    if check:
        want, bound = pa.reference(q, k, v, bounds, D ** -0.5)
        assert bool(((y.double() - want).abs() <= bound).all())
    return st

def cached(D, lens, HQ, weights, check=False):
    g = kv4.gen(2)
    width = -(-max(lens) // 32)
    cache = kv4.make_cache(g, len(lens) * width, 2, 32, D)
    table = kv4.table_of(g, lens, 32, width, len(lens) * width)
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = kv4.rn(g, len(lens), HQ, D).to(torch.bfloat16)
    y = torch.empty_like(q)
    w = torch.zeros(len(lens) * width, 2, 32, device="cuda") if weights else None
    ws = fb.new_kv4_workspace(len(lens), 1, HQ, 2, D, width * 32, weights)
    fb.fp8bq_kv4_attention(q, cache, table, lens_d, y, ws, weights=w)
    st = fb.fp8bq_poll_status(ws)
    if check:
        want, bound, _, _ = kv4.reference(q, cache, table, lens_d, 1, 32, D ** -0.5)
        assert bool(((y.double() - want).abs() <= bound).all())
    return st

# six injected launches
res["prompt_128"] = prompt(128, [700, 90])
res["prompt_64"] = prompt(64, [300])
res["cache_128"] = cached(128, [3000, 200], 8, False)
res["cache_64_weights"] = cached(64, [900, 1], 8, True)
res["cache_256_rows"] = cached(256, [500], 24, False)
res["cache_many_items"] = cached(128, [20] * 100, 8, False)
torch.cuda.synchronize()
# the injection is spent
res["after"] = [prompt(128, [700, 90], True), prompt(64, [300], True),
                cached(128, [3000, 200], 8, False, True), cached(64, [900, 1], 8, True, True),
                cached(256, [500], 24, False, True), cached(128, [20] * 100, 8, False, True)]
print("RESULT " + json.dumps(res))
"""


def test_bounded_waits_report_timeout_and_leave_the_context_usable():
    env = dict(os.environ)
    env["FP8BQ_FAULT_INJECT"] = "skip_first_load:6"
    env["FP8BQ_WAIT_LIMIT_MS"] = "50"
    env["PYTHONPATH"] = os.pathsep.join([ROOT, os.path.join(ROOT, "tests"),
                                         env.get("PYTHONPATH", "")])
    p = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, capture_output=True,
                       text=True, timeout=300)
    assert p.returncode == 0, p.stdout[-2000:] + p.stderr[-4000:]
    line = [l for l in p.stdout.splitlines() if l.startswith("RESULT ")][-1]
    res = json.loads(line[len("RESULT "):])
    after = res.pop("after")
    assert all(v == 8 for v in res.values()), res  # FP8BQ_ERR_TIMEOUT
    assert after == [0] * 6, after
