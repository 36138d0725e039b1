"""Values that are not finite in a prompt: each row gets those that it sees, in their place,
and a call that meets them is not much slower for it."""
import math

import pytest
import torch

import block_wise_fp8_gb300 as fb
from test_gpu_prompt_attention import BF16, I32, check, packed, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("HQ,HK,D", [(2, 2, 128), (2, 2, 48), (6, 2, 64), (16, 2, 128), (128, 1, 32)])
@pytest.mark.parametrize("share", [0.0005, 0.02, 1.0])
def test_rows_get_what_they_see(HQ, HK, D, share):
    """A share of the values, on both sides of the tiles' borders, NaN or one of the infinities:
    infinities of one sign stay that, of both signs make NaN."""
    g = torch.Generator("cuda").manual_seed(HQ + D)
    bounds = [0, 300, 301, 431, 521]
    q, k, v = packed(g, bounds[-1], HQ, HK, D)
    kind = torch.randint(0, 12, v.shape, generator=g, device="cuda")
    kind[torch.rand(v.shape, generator=g, device="cuda") >= share] = 12
    for t in (0, 31, 32, 127, 128, 129, 255, 256, 299, 300, 450):
        kind[t, t % HK, t % D] = 1
    bad = v.clone()
    for i, x in enumerate((math.inf, -math.inf, math.nan, math.inf, math.inf)):
        bad[kind == i] = x
    want, bound = reference(q, k, torch.where(bad.isfinite(), v, 0.0), bounds, D ** -0.5)

    def seen(x):  # by each row and head, within its sequence
        parts = [x[a:b].long().cummax(0).values for a, b in zip(bounds, bounds[1:])]
        return torch.cat(parts).bool().repeat_interleave(HQ // HK, 1)

    up, down, nan = seen(bad == math.inf), seen(bad == -math.inf), seen(bad.isnan())
    nan |= up & down
    off = torch.tensor(bounds, dtype=I32, device="cuda")
    y = torch.empty_like(want, dtype=BF16)
    ws = fb.new_workspace(fb.OP_PROMPT_ATTENTION, bounds[-1], HQ, D)
    fb.fp8bq_prompt_attention(q, k, bad, off, y, ws)
    y = y.double()
    assert bool((up | down).any()) and (share < 0.01 or bool(nan.any()))
    assert bool(y[nan].isnan().all())
    assert bool((y[up & ~nan] == math.inf).all()) and bool((y[down & ~nan] == -math.inf).all())
    fine = ~(nan | up | down)
    check(y[fine], want[fine], bound[fine])


@pytest.mark.parametrize("T,HQ,HK,D", [(4096, 32, 4, 128), (4096, 32, 32, 128), (4096, 12, 4, 64)])
def test_time_with_bad_values(T, HQ, HK, D):
    """A row takes up the tokens that are marked, eight values at a time, until it has nothing
    but NaN: one such value costs little (1.06 times the time without), NaN throughout at most
    1.6 times, infinities throughout 11 to 38 times."""
    g = torch.Generator("cuda").manual_seed(1)
    q, k, v = [torch.randn(T, h, D, generator=g, device="cuda").to(BF16) for h in (HQ, HK, HK)]
    off = torch.tensor([0, T], dtype=I32, device="cuda")
    y = torch.empty_like(q)
    ws = fb.new_workspace(fb.OP_PROMPT_ATTENTION, T, HQ, D)

    def best():
        times = []
        for _ in range(8):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            for _ in range(4):
                fb.fp8bq_prompt_attention(q, k, v, off, y, ws)
            end.record()
            torch.cuda.synchronize()
            times.append(start.elapsed_time(end) / 4)
        return min(times)

    plain = best()
    v[T // 2, 0, 3] = math.nan
    one = best()
    v.fill_(math.inf)
    infinite = best()
    v.fill_(math.nan)
    full = best()
    assert fb.fp8bq_poll_status(ws) == 0
    print(f"{plain * 1e3:.1f} us; one NaN {one * 1e3:.1f}, infinite {infinite * 1e3:.1f}, NaN {full * 1e3:.1f}")
    assert one < 4 * plain and full < 12 * plain and infinite < 60 * plain


def test_marks_of_one_unit_and_the_next():
    """Many units a CTA, a few of them with values that are not finite, far apart in time for
    the rows of a warp (some have none to take up, some 256): nothing is lost or left behind."""
    HQ, HK, D = 24, 24, 64
    g = torch.Generator("cuda").manual_seed(4)
    T = 1500
    q, k, v = packed(g, T, HQ, HK, D)
    bounds = [0, 700, 701, 1100, T]
    bad = v.clone()
    for i in range(60):
        t, h = (i * 97 + 11) % T, i % HK
        bad[t, h, (5 * i) % D:] = math.inf
        bad[t, h, :(3 * i) % 9] = math.nan
    off = torch.tensor(bounds, dtype=I32, device="cuda")
    ws = fb.new_workspace(fb.OP_PROMPT_ATTENTION, T, HQ, D)
    want, bound = reference(q, k, torch.where(bad.isfinite(), v, 0.0), bounds, D ** -0.5)

    def seen(x):
        return torch.cat([x[a:b].long().cummax(0).values for a, b in zip(bounds, bounds[1:])]).bool()

    nan, inf = seen(bad.isnan()), seen(bad == math.inf)
    for _ in range(20):
        y = torch.empty_like(want, dtype=BF16)
        fb.fp8bq_prompt_attention(q, k, bad, off, y, ws)
        y = y.double()
        assert bool(y[nan].isnan().all()) and bool((y[inf & ~nan] == math.inf).all())
        check(y[~(nan | inf)], want[~(nan | inf)], bound[~(nan | inf)])
