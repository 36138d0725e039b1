"""Attention over the 4-bit cache where scores are large: the parts of a row that several
warps and CTAs hold have to be joined as exactly as the scores within one are compared."""
import pytest
import torch

import block_wise_fp8_gb300 as fb
from test_gpu_kv4 import BF16, I32, gen, make_cache, parts, rn, rows, table_of, values

pytestmark = pytest.mark.gpu


def attend(q, cache, table, lens, page, Tq=1, scale=None):
    """y and the weights added, [pages, HK, page]."""
    N, HQ, D = q.shape
    w = torch.zeros(cache.shape[0], cache.shape[1], page, device="cuda")
    y = torch.empty_like(q)
    ws = fb.new_kv4_workspace(N // Tq, Tq, HQ, cache.shape[1], D, table.shape[1] * page, True)
    fb.fp8bq_kv4_attention(q, cache, table, lens, y, ws, weights=w, scale=scale)
    assert fb.fp8bq_poll_status(ws) == 0
    without = torch.empty_like(q)
    fb.fp8bq_kv4_attention(q, cache, table, lens, without, ws, scale=scale)
    assert torch.equal(without.view(torch.int16), y.view(torch.int16))
    return y, w


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,HQ", [([40], 1), ([700], 8), ([20000, 333], 3), ([9000, 130], 12)])
def test_close_scores_far_from_zero(D, lens, HQ):
    """Scores q0 * 2688 + c with q0 = 1024 and c a code of -6 .. 6 that the tokens of a block
    of 32 share: FP32 holds every partial sum (multiples of 1/2 below 2^22), so that what is
    left of a score's error is the exponential's argument (differences up to 12, times a
    scale in FP32: 2^-22 of 12 * 0.5 * log2 e) and value (2^-21).  The weights' error is that
    of the arguments and of the sums over n tokens, (n / 8 + 64) steps of 2^-23; the output's
    has half a step of FP16 for each weight, 2^-25 of the largest, and half one of BF16."""
    page, B, scale = 64, len(lens), 0.5
    g = gen(D + HQ)
    width = -(-max(lens) // page)
    cache = make_cache(g, B * width, 1, page, D)
    table = table_of(g, lens, page, width, B * width)
    kc, ks = parts(cache, page, D)[:2]
    kc.zero_()
    kc[..., 0] = 7                       # 6 * 448 in place 0
    ks[..., 0], ks[..., 1] = 0x7E, 0x38  # 448, 1
    for b, n in enumerate(lens):
        t = torch.arange(n, device="cuda")
        block = t // 32
        code = (block * 5 + 3) % 8 + 8 * (block * 3 % 2)
        kc[table[b].long()[t // page], 0, t % page, 8] = code.to(torch.uint8)  # place 16
    lens_d = torch.tensor(lens, dtype=I32, device="cuda")
    q = torch.zeros(B, HQ, D, dtype=BF16, device="cuda")
    q[:, :, 0], q[:, :, 16] = 1024.0, 1.0
    y, w = attend(q, cache, table, lens_d, page, scale=scale)
    p4 = parts(cache, page, D)
    for b, n in enumerate(lens):
        k, v = [values(rows(p4[i], table, b, n, page)[0], rows(p4[i + 1], table, b, n, page)[0])[0]
                for i in (0, 2)]
        s = (k @ q[b, 0].double()) * scale
        assert float(s.min()) > 1.3e6
        p = torch.softmax(s, 0)
        ds = 12 * scale * 1.4427 * 2.0 ** -22 + 2.0 ** -21
        sums = (n / 8 + 64) * 2.0 ** -23
        want, size = p @ v, p @ v.abs()
        bound = (want.abs() * 2.0 ** -8 + size * (2.0 ** -11 + 2 * ds + 2 * sums) * 1.01 +
                 v.abs().sum(0) * 2.0 ** -25)
        assert bool(((y[b].double() - want).abs() <= bound).all()), (
            b, float(((y[b].double() - want).abs() / bound).max()))
        t = torch.arange(n, device="cuda")
        got = w[table[b].long()[t // page], 0, t % page].double()
        assert bool(((got - HQ * p).abs() <= HQ * p * (2 * ds + 2 * sums + HQ * 2.0 ** -23)).all())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,Tq,HQ,HK", [([200], 1, 8, 1), ([1], 1, 8, 1), ([20000, 333], 1, 8, 1),
                                           ([1000, 9000], 2, 24, 2)])
@pytest.mark.parametrize("sign", [0, 1, -1])
def test_one_token_has_all_the_weight(D, lens, Tq, HQ, HK, sign):
    """Queries of 1e5 to 3e37: scores pass FP32's range, in either direction (sign: all of
    them positive, or negative), and the largest one's token has the whole weight: its value
    comes out exactly, and its weight grows by 1."""
    page, B = 32, len(lens)
    g = gen(D + HQ + len(lens))
    width = -(-max(lens) // page)
    cache = make_cache(g, B * width, HK, page, D)
    kc = parts(cache, page, D)[0]
    if sign:
        kc.copy_(kc & 0x77)
    table = table_of(g, lens, page, width, B * width)
    lens_d = torch.tensor(lens, dtype=I32, device="cuda")
    q = rn(g, B * Tq, HQ, D)
    if sign:
        q = sign * (q.abs() + 0.01)
    size = torch.tensor([1e5, 1e12, 1e30, 3e37], device="cuda")[torch.arange(HQ, device="cuda") % 4]
    q = (q.clamp(-8, 8) * size[:, None]).to(BF16)
    y, w = attend(q, cache, table, lens_d, page, Tq)
    assert bool(y.isfinite().all()) and bool(w.isfinite().all())
    p4 = parts(cache, page, D)
    G, total, clear_rows = HQ // HK, torch.zeros_like(w, dtype=torch.float64), 0
    for b, n in enumerate(lens):
        k, v = [values(rows(p4[i], table, b, n, page)[0], rows(p4[i + 1], table, b, n, page)[0])
                for i in (0, 2)]
        for i in range(Tq):
            m = n - (Tq - 1 - i)
            qd = q[b * Tq + i].double().view(HK, G, D)
            s = torch.einsum("hgd,hnd->hgn", qd, k[:, :m])
            mag = torch.einsum("hgd,hnd->hgn", qd.abs(), k[:, :m].abs()).amax(-1)
            top = s.topk(min(2, m), -1)
            # FP32 sums of D products cannot turn which of the two is larger, and e^-200 of
            # the other is nothing
            clear = torch.ones(HK, G, dtype=torch.bool, device="cuda")
            if m > 1:
                clear = top.values[..., 0] - top.values[..., 1] > mag * (D + 8) * 2.0 ** -22 + 200 * D ** 0.5
            want = v.gather(1, top.indices[..., 0, None].expand(-1, -1, D))
            got = y[b * Tq + i].double().view(HK, G, D)
            assert torch.equal(got[clear], want[clear])
            clear_rows += int(clear.sum())
            if bool(clear.all()) and B * Tq == 1:
                t = top.indices[0, :, 0]
                total.index_put_((table[b].long()[t // page], torch.zeros_like(t), t % page),
                                 torch.ones(G, dtype=torch.float64, device="cuda"), accumulate=True)
                assert torch.equal(w.double(), total)
    assert clear_rows > 0.8 * B * Tq * HQ
    # every row gives out 1, to (n / 8 + 64) steps of 2^-23
    assert abs(float(w.double().sum()) - B * Tq * HQ) <= B * Tq * HQ * (max(lens) / 8 + 64) * 2.0 ** -22


def test_scale_and_query_both_large():
    """A scale of 1e30 on top of queries of 1e30: their product passes FP32's range."""
    page, D = 64, 128
    g = gen(5)
    cache = make_cache(g, 12, 1, page, D)
    table = torch.arange(12, device="cuda", dtype=I32)[None]
    lens = torch.tensor([700], dtype=I32, device="cuda")
    q = (rn(g, 1, 4, D) * 1e30).to(BF16)
    y, w = attend(q, cache, table, lens, page, scale=1e30)
    p4 = parts(cache, page, D)
    k, v = [values(rows(p4[i], table, 0, 700, page)[0], rows(p4[i + 1], table, 0, 700, page)[0])[0]
            for i in (0, 2)]
    best = (q[0].double() @ k.t()).argmax(-1)
    assert torch.equal(y[0].double(), v[best])
    assert float(w.sum()) == 4.0
