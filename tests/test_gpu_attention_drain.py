"""A block of the attention kernels that gives up waiting keeps its memory until its copies in
flight have landed: the next launch, behind it in the stream without a pause, gets the same
memory and is right.  One copy that never lands, as in test_gpu_attention_fault.py: of a
prompt's first unit (the queries' copies are on their way by then), and of a cached sequence
of one tile (the copying warp has nothing left to issue when the others give up)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys
import torch
import block_wise_fp8_gb300 as fb
import test_gpu_kv4 as kv4
import test_gpu_prompt_attention as pa

kind, D, lens, HQ, HK, weights = eval(sys.argv[1])
g = kv4.gen(1)
I32 = torch.int32
if kind == "prompt":
    bounds = [0]
    for n in lens:
        bounds.append(bounds[-1] + n)
    q, k, v = pa.packed(g, bounds[-1], HQ, HK, D)
    off = torch.tensor(bounds, dtype=I32, device="cuda")
    spaces = [fb.new_workspace(fb.OP_PROMPT_ATTENTION, bounds[-1], HQ, D) for _ in range(2)]
    ys = [torch.empty_like(q.contiguous()) for _ in range(2)]
    call = lambda i: fb.fp8bq_prompt_attention(q, k, v, off, ys[i], spaces[i])
    want, bound = pa.reference(q, k, v, bounds, D ** -0.5)
else:
    width = -(-max(lens) // 32)
    cache = kv4.make_cache(g, len(lens) * width, HK, 32, D)
    table = kv4.table_of(g, lens, 32, width, len(lens) * width)
    lens_d = torch.tensor(lens, dtype=I32, device="cuda")
    q = kv4.rn(g, len(lens), HQ, D).to(torch.bfloat16)
    w = torch.zeros(len(lens) * width, HK, 32, device="cuda") if weights else None
    spaces = [fb.new_kv4_workspace(len(lens), 1, HQ, HK, D, width * 32, weights) for _ in range(2)]
    ys = [torch.empty_like(q) for _ in range(2)]
    call = lambda i: fb.fp8bq_kv4_attention(q, cache, table, lens_d, ys[i], spaces[i], weights=w)
    want, bound, _, _ = kv4.reference(q, cache, table, lens_d, 1, 32, D ** -0.5)
torch.cuda.synchronize()
call(0)  # its wait runs out
call(1)
torch.cuda.synchronize()
assert [fb.fp8bq_poll_status(s) for s in spaces] == [8, 0]
assert bool(((ys[1].double() - want).abs() <= bound).all())
"""


@pytest.mark.parametrize("case", [
    ("prompt", 128, [700, 90, 333], 32, 8, False), ("prompt", 64, [2000, 300], 24, 8, False),
    ("prompt", 128, [5], 1, 1, False), ("cache", 128, [40], 8, 1, False),
    ("cache", 64, [900, 1], 8, 2, True), ("cache", 256, [500] * 40, 24, 2, False)])
def test_the_next_launch_is_right(case):
    env = dict(os.environ)
    env["FP8BQ_FAULT_INJECT"] = "skip_first_load:1"
    env["FP8BQ_WAIT_LIMIT_MS"] = "50"
    env["PYTHONPATH"] = os.pathsep.join([ROOT, os.path.join(ROOT, "tests"),
                                         env.get("PYTHONPATH", "")])
    p = subprocess.run([sys.executable, "-c", CHILD, repr(case)], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stdout[-2000:] + p.stderr[-4000:]
