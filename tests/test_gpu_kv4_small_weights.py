"""Attention over the 4-bit cache where one early token draws nearly all of a row's weight and
has little to say: what is left of the output is the sum of many small weights."""
import pytest
import torch

import block_wise_fp8_gb300 as fb
from test_gpu_kv4 import BF16, I32, gen, make_cache, parts, rows, table_of, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,HQ", [(64, 1), (128, 8), (128, 16), (256, 4)])
@pytest.mark.parametrize("n,at", [(300, 0), (5000, 3), (70000, 69)])
@pytest.mark.parametrize("gap", [24, 27, 30])
def test_a_token_with_nearly_all_the_weight(D, HQ, n, at, gap):
    """The others' weights are 2^-gap of its, its value is zero, theirs are positive.  Scores
    are exact (q0 * 448 * code), the exponents' arguments below 32 (2^-23 of them), a weight in
    FP16 has half a step, 2^-11 of it or 2^-32 of the row's largest; its value and the sums of
    n tokens as elsewhere, (n / 8 + 64) steps of 2^-23; BF16 2^-8."""
    page = 64
    g = gen(n + D)
    width = -(-n // page)
    cache = make_cache(g, width, 1, page, D)
    table = table_of(g, [n], page, width, width)
    kc, ks, vc, _ = parts(cache, page, D)
    kc.zero_()
    ks[..., 0] = 0x7E                                      # 448
    kc[table[0, at // page].long(), 0, at % page, 0] = 2   # a code of 1; the others' are 0
    vc.copy_(vc & 0x77 | 0x11)
    vc[table[0, at // page].long(), 0, at % page] = 0
    q = torch.zeros(1, HQ, D, dtype=BF16, device="cuda")
    q[..., 0] = 1.0
    scale = gap * 0.6931471805599453 / 448
    lens = torch.tensor([n], dtype=I32, device="cuda")
    y = torch.empty_like(q)
    w = torch.zeros(width, 1, page, device="cuda")
    ws = fb.new_kv4_workspace(1, 1, HQ, 1, D, width * page, True)
    fb.fp8bq_kv4_attention(q, cache, table, lens, y, ws, weights=w, scale=scale)
    p4 = parts(cache, page, D)
    k, v = [values(rows(p4[i], table, 0, n, page)[0], rows(p4[i + 1], table, 0, n, page)[0])[0]
            for i in (0, 2)]
    p = torch.softmax(k @ q[0, 0].double() * scale, 0)
    want = p @ v
    ds, sums = 32 * 2.0 ** -23 + 2.0 ** -21, (n / 8 + 64) * 2.0 ** -23
    bound = want * (2.0 ** -8 + (2.0 ** -11 + 2 * ds + 2 * sums) * 1.01) + v.sum(0) * 2.0 ** -32
    err = (y[0].double() - want).abs()
    assert float(want.min()) > 0
    assert bool((err <= bound).all()), float((err / want).max())
    t = torch.arange(n, device="cuda")
    got = w[table[0].long()[t // page], 0, t % page].double()
    assert bool(((got - HQ * p).abs() <= HQ * p * (2 * ds + 2 * sums + HQ * 2.0 ** -23)).all())
