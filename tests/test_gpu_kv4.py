"""The 4-bit paged cache and the attention over it, against plain forms in 64 bits.

Written codes and scales are bit-exact.  Attention: a row's bound is derived from
  half a step of BF16 (2^-8) for the output,
  half a step of FP16 for each weight: 2^-11 of it, and 2^-25 of the largest,
  the scores: products of D exact terms summed in FP32 (D + 8 steps of 2^-23 of the
  sum of magnitudes: tensor cores may truncate), times the scale, and the rounding
  of an exponential's argument (2^-23 of it) and value (2^-22),
  sums over n tokens in FP32, (n / 8 + 64) steps of 2^-23."""
import math

import pytest
import torch

import block_wise_fp8_gb300 as fb
from gpu_util import Guarded

pytestmark = pytest.mark.gpu
BF16, F32, I32, I64, U8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8
GRID = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
SCALES = torch.tensor([m * 2.0 ** -9 for m in range(8)] +
                      [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1],
                      dtype=torch.float64)  # in the order of their codes


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def rn(g, *s):
    return torch.randn(*s, generator=g, device="cuda")


def nearest(x, grid):
    """Index in `grid` of the nearest entry, ties to the even index; beyond its end the last."""
    grid = grid.to(x.device)
    lo = (torch.bucketize(x, grid, right=True) - 1).clamp(0, len(grid) - 2)
    down, up = x - grid[lo], grid[lo + 1] - x
    return lo + torch.where(down == up, lo % 2 == 1, down > up).long()


def quantise(x, inv=1.0):
    """codes [..., D/2] and scale codes [..., D/16] of BF16 x [..., D], by the formula in 64
    bits (the product with inv and the scale's division in binary32, as the interface says)."""
    x = (x.float() * inv).unflatten(-1, (-1, 16))
    amax = x.abs().amax(-1)
    si = nearest((amax / 6.0).double().clamp(max=448.0), SCALES).clamp(min=1)
    s = SCALES.to(x.device)[si]
    c = nearest((x.double().abs() / s[..., None]).clamp(max=6.0), GRID)
    c = (c + 8 * torch.signbit(x).long()).flatten(-2)
    return (c[..., 0::2] + 16 * c[..., 1::2]).to(U8), si.to(U8)


def values(codes, scales):
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    v = GRID.to(codes.device)[nib % 8] * torch.where(nib >= 8, -1.0, 1.0)
    s = scales.contiguous().view(torch.float8_e4m3fn).double()
    return v * s.repeat_interleave(16, -1)


def parts(cache, page, D):
    c, s = page * D // 2, page * D // 16
    return [p.unflatten(-1, (page, -1)) for p in cache.split([c, s, c, s], -1)]


def make_cache(g, pages, HK, page, D):
    """A cache of random codes and scales; the scales' magnitudes in [2^-3, 2^1)."""
    cache = torch.randint(0, 256, (pages, HK, page * 9 * D // 8), generator=g, device="cuda",
                          dtype=torch.int64).to(U8)
    for i in (1, 3):
        p = parts(cache, page, D)[i]
        p.copy_((torch.randint(4 * 8, 8 * 8, p.shape, generator=g, device="cuda")).to(U8))
    return cache


def rows(x, table, b, n, page):
    """Entries [HK, n, ...] of sequence b's first n tokens, and which of them are there."""
    t = torch.arange(n, device="cuda")
    pg = table[b].long()[t // page]
    there = (pg >= 0) & (pg < x.shape[0])
    return x[pg.clamp(0, x.shape[0] - 1), :, t % page].transpose(0, 1), there


# ---------------------------------------------------------------- append and read

@pytest.mark.parametrize("T,HK,D,page,bits", [(1, 1, 64, 16, 32), (3, 2, 128, 16, 64),
                                              (67, 3, 128, 64, 32), (130, 8, 256, 128, 64),
                                              (1025, 4, 64, 32, 64)])
def test_append_and_read(T, HK, D, page, bits):
    g = gen(T + D)
    pages = 2 * -(-T // page) + 1
    k = rn(g, T, HK, D) * torch.exp2(torch.randint(-20, 12, (T, HK, 1), generator=g, device="cuda"))
    qkv = torch.zeros(T, (2 * HK + 1) * D, dtype=BF16, device="cuda")
    kv, vv = qkv[:, D:(HK + 1) * D].view(T, HK, D), qkv[:, (HK + 1) * D:].view(T, HK, D)
    kv.copy_(k), vv.copy_(rn(g, T, HK, D))
    kv[0, 0, :32] = 0.0
    kv[0, 0, 16] = -0.0
    kv[-1, -1, 16:32] = 2.0 ** -20
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].to(I64 if bits == 64 else I32)
    drop = torch.rand(T, generator=g, device="cuda") < 0.2
    slots[drop] = torch.tensor([-1, pages * page, -7], device="cuda", dtype=slots.dtype)[
        torch.arange(int(drop.sum()), device="cuda") % 3]
    guard = Guarded((pages, HK, page * 9 * D // 8), U8, fill=0x5A)
    weights = torch.full((pages, HK, page), 3.0, device="cuda")
    want = guard.t.clone()
    w = parts(want, page, D)
    on = ~drop
    at = slots[on].long()
    for i, x in ((0, kv), (2, vv)):
        codes, sc = quantise(x[on])
        w[i][at // page, :, at % page] = codes
        w[i + 1][at // page, :, at % page] = sc
    fb.fp8bq_kv4_append(kv, vv, slots, guard.t, weights)
    guard.check("cache")
    assert torch.equal(guard.t, want)
    want_w = torch.full_like(weights, 3.0)
    want_w[at // page, :, at % page] = 0.0
    assert torch.equal(weights, want_w)
    ko, vo = (Guarded((T, HK, D), BF16, fill=9.0) for _ in range(2))
    fb.fp8bq_kv4_read(guard.t, slots, ko.t, vo.t)
    for o, i in ((ko, 0), (vo, 2)):
        o.check("rows")
        exact = torch.full((T, HK, D), 9.0, dtype=torch.float64, device="cuda")
        exact[on] = values(w[i][at // page, :, at % page], w[i + 1][at // page, :, at % page])
        assert torch.equal(o.t.double(), exact)


def test_append_every_bf16():
    """Every finite BF16 value below each of a row of group maxima, on both sides."""
    mags = torch.arange(0, 0x7F80, dtype=torch.int32).to(torch.int16).view(BF16)
    x = torch.cat([mags, -mags]).cuda()
    for top in (0.0117, 1.0, 5.25, 6.0, 448.0, 2687.0, 2689.0, 3e38, 1e-3, 2.0 ** -9, 1.1e-4):
        v = x[x.abs() <= top]
        n = -(-v.numel() // 15)
        rowsx = torch.zeros(n * 15, dtype=BF16, device="cuda")
        rowsx[:v.numel()] = v
        rowsx = torch.cat([torch.full((n, 1), top, dtype=BF16, device="cuda"), rowsx.view(n, 15)], 1)
        T = -(-n // 4)
        k = torch.zeros(T * 4, 16, dtype=BF16, device="cuda")
        k[:n] = rowsx
        k = k.view(T, 1, 64)
        pages = -(-T // 128)
        cache = fb.new_kv4_cache(pages, 1, 128, 64)
        fb.fp8bq_kv4_append(k, -k, torch.arange(T, device="cuda"), cache)
        p = parts(cache, 128, 64)
        at = torch.arange(T, device="cuda")
        for i, y in ((0, k), (2, -k)):
            codes, sc = quantise(y)
            assert torch.equal(p[i + 1][at // 128, :, at % 128], sc), top
            assert torch.equal(p[i][at // 128, :, at % 128], codes), top


def test_append_every_scale():
    """Groups whose maxima give every scale that there is, values at and beside every tie
    of the codes: the nearest code of the exact quotient."""
    s = SCALES[1:].float()
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    x = torch.zeros(len(s), 2, 16)
    x[:, :, 0] = (s * 6.0)[:, None]
    x[:, 0, 1:8] = s[:, None] * ties
    x[:, 1, 1:8] = -s[:, None] * ties
    up = x[:, 0, 1:8].to(BF16).view(torch.int16)
    x[:, 0, 8:15] = (up + 1).view(BF16).float()
    x[:, 1, 8:15] = -(up - 1).view(BF16).float()
    k = torch.zeros(len(s), 1, 64)
    k[:, 0, :32] = x.view(len(s), 32)
    k[:, 0, 32:] = -x.view(len(s), 32)
    k = k.to(BF16).cuda()
    at = torch.arange(len(s), device="cuda")
    cache = fb.new_kv4_cache(-(-len(s) // 64), 1, 64, 64)
    fb.fp8bq_kv4_append(k, -k, at, cache)
    p = parts(cache, 64, 64)
    for i, y in ((0, k), (2, -k)):
        codes, sc = quantise(y)
        assert torch.equal(p[i + 1][at // 64, :, at % 64], sc)
        assert torch.equal(p[i][at // 64, :, at % 64], codes)
    assert len(sc.unique()) == len(s)  # every scale was met


def test_append_special_values():
    inf, nan = math.inf, math.nan
    k = torch.zeros(4, 1, 64, dtype=BF16, device="cuda")
    k[0, 0, :4] = torch.tensor([inf, -inf, 5.0, 1000.0])
    k[1, 0, 16:18] = torch.tensor([nan, 3.0])
    k[2, 0, :2] = torch.tensor([inf, nan])
    cache = fb.new_kv4_cache(1, 1, 16, 64)
    fb.fp8bq_kv4_append(k, k, torch.arange(4, device="cuda"), cache)
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    fb.fp8bq_kv4_read(cache, torch.arange(4, device="cuda"), ko, vo)
    assert torch.equal(torch.nan_to_num(ko, nan=7.0), torch.nan_to_num(vo, nan=7.0))
    # 1000 / 448 = 2.23 is nearest to 2
    assert ko[0, 0, :4].tolist() == [2688.0, -2688.0, 0.0, 896.0]
    assert bool(ko[1, 0, 16:32].isnan().all()) and bool(ko[2, 0, :16].isnan().all())
    clean = torch.cat([ko[0, 0, 4:], ko[1, 0, :16], ko[1, 0, 32:], ko[2, 0, 16:], ko[3, 0]])
    assert bool((clean == 0).all())


@pytest.mark.parametrize("ks,vs", [(0.25, 8.0), (0.3, 1.7)])
def test_append_scales(ks, vs):
    g = gen(5)
    k, v = rn(g, 33, 2, 128).to(BF16), rn(g, 33, 2, 128).to(BF16)
    cache = fb.new_kv4_cache(3, 2, 16, 128)
    at = torch.arange(33, device="cuda")
    fb.fp8bq_kv4_append(k, v, at, cache, k_scale=ks, v_scale=vs)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    fb.fp8bq_kv4_read(cache, at, ko, vo, k_scale=ks, v_scale=vs)
    p = parts(cache, 16, 128)
    for i, x, o, s in ((0, k, ko, ks), (2, v, vo, vs)):
        s32 = torch.tensor(s, dtype=F32)
        codes, sc = quantise(x, float(torch.tensor(1.0) / s32))
        assert torch.equal(p[i][at // 16, :, at % 16], codes)
        assert torch.equal(p[i + 1][at // 16, :, at % 16], sc)
        exact = values(codes, sc) * float(s32)
        # one product in FP32 (2^-24) and one rounding to BF16 (2^-8)
        assert bool(((o.double() - exact).abs() <= exact.abs() * (2.0 ** -8 + 2.0 ** -23)).all())


# ---------------------------------------------------------------- attention

def reference(q, cache, table, lens, Tq, page, scale, ks=1.0, vs=1.0):
    """(y, bound, weights added, their bound) in 64 bits, row by row."""
    N, HQ, D = q.shape
    B, HK = N // Tq, cache.shape[1]
    G = HQ // HK
    pages = cache.shape[0]
    p4 = parts(cache, page, D)
    y = torch.zeros(N, HQ, D, dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(y)
    add = torch.zeros(pages, HK, page, dtype=torch.float64, device="cuda")
    add_b = torch.zeros_like(add)
    longest = table.shape[1] * page
    for b in range(B):
        n = min(max(int(lens[b]), 0), longest)
        if n == 0:
            continue
        kc, there = rows(p4[0], table, b, n, page)
        k = values(kc, rows(p4[1], table, b, n, page)[0]) * ks
        v = values(rows(p4[2], table, b, n, page)[0], rows(p4[3], table, b, n, page)[0]) * vs
        t = torch.arange(n, device="cuda")
        for i in range(Tq):
            m = n - (Tq - 1 - i)
            see = there & (t < m)
            if not bool(see.any()):
                continue
            qd = q[b * Tq + i].double().view(HK, G, D)
            kk, vv = k[:, see], v[:, see]
            s = torch.einsum("hgd,hnd->hgn", qd, kk) * scale
            mag = torch.einsum("hgd,hnd->hgn", qd.abs(), kk.abs()) * scale
            p = torch.softmax(s, -1)
            out = torch.einsum("hgn,hnd->hgd", p, vv)
            size = torch.einsum("hgn,hnd->hgd", p, vv.abs())
            ds = (mag.amax(-1) * (D + 8) * 2.0 ** -23 + s.abs().amax(-1) * 2.0 ** -22 + 2.0 ** -21)
            sums = (m / 8 + 64) * 2.0 ** -23
            rel = (2.0 ** -11 + 2 * ds + 2 * sums)[..., None]
            y[b * Tq + i] = out.reshape(HQ, D)
            bd = out.abs() * 2.0 ** -8 + size * rel * 1.01 + vv.abs().sum(1)[:, None] * 2.0 ** -25
            bound[b * Tq + i] = bd.reshape(HQ, D)
            tt = t[see]
            pg = table[b].long()[tt // page]
            add[pg, :, tt % page] += p.sum(1).t()
            add_b[pg, :, tt % page] += (p * (2 * ds + 2 * sums)[..., None]).sum(1).t()
    return y, bound, add, add_b


def table_of(g, lens, page, width, pages):
    order = torch.randperm(pages, generator=g, device="cuda").to(I32)
    table = torch.full((len(lens), width), -1, dtype=I32, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        need = min(width, -(-max(0, n) // page))
        table[b, :need] = order[at:at + need]
        at += need
    assert at <= pages
    return table


def attend(lens, Tq, HQ, HK, D, page, seed=0, weights=True, width=None, ks=1.0, vs=1.0, scale=None,
           edit=None, strided=True):
    g = gen(seed)
    B = len(lens)
    width = width or max(1, max(-(-max(0, n) // page) for n in lens))
    pages = B * width + 2
    cache = make_cache(g, pages, HK, page, D)
    table = table_of(g, lens, page, width, pages)
    if edit:
        edit(cache, table)
    lens_d = torch.tensor(lens, dtype=I32, device="cuda")
    base = rn(g, B * Tq, (HQ + 3) * D).to(BF16)
    q = base[:, 2 * D:(HQ + 2) * D].view(B * Tq, HQ, D) if strided else base[:, :HQ * D].reshape(B * Tq, HQ, D)
    sc = D ** -0.5 if scale is None else scale
    y = Guarded((B * Tq, HQ, D), BF16, fill=5.0)
    w0 = torch.rand(pages, HK, page, generator=g, device="cuda") if weights else None
    w = w0.clone() if weights else None
    size = fb.fp8bq_kv4_workspace_bytes(B, Tq, HQ, HK, D, width * page, weights)
    ws = Guarded((size,), U8, fill=0)
    for again in range(2):
        if weights:
            w.copy_(w0)
        y.t.fill_(5.0)
        fb.fp8bq_kv4_attention(q, cache, table, lens_d, y.t, ws.t, weights=w, scale=scale,
                               k_scale=ks, v_scale=vs)
        assert fb.fp8bq_poll_status(ws.t) == 0
        y.check("y"), ws.check("workspace")
        if again:
            assert torch.equal(first.view(torch.int16), y.t.view(torch.int16))  # NaN too
            assert not weights or torch.equal(first_w, w)
        first, first_w = y.t.clone(), w.clone() if weights else None
    want, bound, add, add_b = reference(q, cache, table, lens_d, Tq, page, sc, ks, vs)
    return y.t.double(), want, bound, w, w0, add, add_b


def check(out, want, bound, w, w0, add, add_b):
    err = (out - want).abs()
    assert bool((err <= bound).all()), f"{float((err / bound.clamp(min=1e-300)).max())} of the bound"
    if w is not None:
        total = w0.double() + add
        assert bool(((w.double() - total).abs() <= add_b + total * 2.0 ** -23).all())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Tq,HQ,HK", [(1, 8, 1), (2, 10, 2), (5, 3, 3)])
def test_attention(D, page, Tq, HQ, HK):
    check(*attend([1, 0, 17, 128, 129, 700, 3, 64], Tq, HQ, HK, D, page, seed=D + page + Tq))


@pytest.mark.parametrize("HQ,HK,Tq", [(1, 1, 1), (16, 1, 1), (24, 1, 1), (64, 4, 2), (128, 1, 1),
                                      (8, 8, 16), (7, 7, 3), (128, 16, 1)])
def test_attention_heads(HQ, HK, Tq):
    check(*attend([33, 1000, 5], Tq, HQ, HK, 128, 32, seed=HQ, weights=Tq != 2))


@pytest.mark.parametrize("lens", [[1], [2], [127], [128], [129], [5000], [40000, 1, 39999],
                                  [1] * 300, [130] * 65, list(range(0, 200, 3))])
def test_attention_lengths(lens):
    check(*attend(lens, 1, 8, 2, 128, 64, seed=len(lens), weights=len(lens) < 5))


def test_attention_scales_and_wider_tables():
    check(*attend([100, 257], 2, 8, 2, 128, 16, ks=0.37, vs=3.0, scale=0.2, width=40))
    check(*attend([100, 257, -5, 10 ** 6], 1, 8, 2, 64, 16, width=20, strided=False))


def test_attention_sharp_rows():
    """Scores far apart: the largest token decides, the others are lost without a trace."""
    check(*attend([3000, 77], 1, 8, 2, 128, 64, scale=3.0))
    check(*attend([3000, 77], 2, 8, 2, 128, 64, scale=1e-4))


def test_bytes_behind_the_end_have_no_part():
    """NaN scales and any codes behind a sequence's end or in pages it does not name."""
    def edit(cache, table):
        seen = torch.zeros(cache.shape[0], dtype=torch.bool, device="cuda")
        seen[table[table >= 0].long()] = True
        cache[~seen] = 0xFF
        p = parts(cache, 32, 128)
        for b, n in enumerate((45, 100, 3)):
            last = int(table[b, (n - 1) // 32])
            for x in p:
                x[last, :, (n - 1) % 32 + 1:] = 0xFF
    check(*attend([45, 100, 3], 1, 8, 2, 128, 32, edit=edit))
    check(*attend([45, 100, 3], 3, 8, 2, 128, 32, edit=edit))


def test_pages_that_are_not_there():
    def edit(cache, table):
        table[0, 1] = -1
        table[1, 0] = cache.shape[0]
        table[2, :] = 2 ** 31 - 1
        table[3, 5] = -2 ** 31
    check(*attend([200, 150, 64, 700], 1, 8, 2, 128, 64, edit=edit))
    check(*attend([200, 150, 64, 700], 2, 16, 2, 128, 16, edit=edit))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_nan_reaches_the_rows_that_see_it(D):
    """A NaN value scale in the last of three new tokens: the last query's values of that
    group alone; a NaN key scale: the whole row of that query alone."""
    n, page = 70, 64
    for part in (1, 3):
        def edit(cache, table):
            parts(cache, page, D)[part][int(table[0, (n - 1) // page]), 0, (n - 1) % page, 1] = 0x7F
        out, want, bound, *_ = attend([n, 50], 3, 4, 2, D, page, weights=False, edit=edit)
        hit = torch.zeros_like(out, dtype=torch.bool)
        if part == 3:
            hit[2, :2, 16:32] = True
        else:
            hit[2, :2] = True
        assert bool(out[hit].isnan().all()) and bool(want[hit].isnan().all())
        assert bool(((out - want).abs() <= bound)[~hit].all())


def test_queries_of_any_size():
    g = gen(8)
    cache = make_cache(g, 4, 1, 64, 128)
    table = torch.arange(4, device="cuda", dtype=I32)[None]
    lens = torch.tensor([200], dtype=I32, device="cuda")
    q = rn(g, 1, 8, 128)
    q[0, 1:] *= torch.tensor([1e-30, 1e30, 1e-38, 0.0, 3e37, 1e-3, 1e3], device="cuda")[:, None]
    q = q.to(BF16)
    y = torch.empty_like(q)
    ws = fb.new_kv4_workspace(1, 1, 8, 1, 128, 256)
    fb.fp8bq_kv4_attention(q, cache, table, lens, y, ws)
    want, bound, _, _ = reference(q, cache, table, lens, 1, 64, 128 ** -0.5)
    ok = [0, 1, 3, 4, 6]
    assert bool(((y.double() - want).abs() <= bound)[:, ok].all())
    assert bool(y[:, [0, 1, 2, 3, 4, 6, 7]].isfinite().all())  # scores of 1e30 pick one token
    q[0, 0, 5] = math.nan
    q[0, 1, 5] = math.inf
    fb.fp8bq_kv4_attention(q, cache, table, lens, y, ws)
    assert bool(y[0, :2].isnan().all()) and bool(y[0, 3:5].isfinite().all())


def test_attention_offsets_past_32_bits():
    """Pages whose byte offset lies beyond 2^32."""
    g = gen(3)
    page, HK, D = 128, 8, 128
    pages = 2 ** 32 // (HK * page * 9 * D // 8) + 40
    cache = torch.zeros(pages, HK, page * 9 * D // 8, dtype=U8, device="cuda")
    few = make_cache(g, 8, HK, page, D)
    at = torch.tensor([pages - 1, 3, pages - 9, pages - 30, 0, pages - 2, 7, pages - 12], device="cuda")
    cache[at] = few
    table = at.view(2, 4).to(I32)
    lens = torch.tensor([500, 390], dtype=I32, device="cuda")
    q = rn(g, 2, 16, D).to(BF16)
    y, y2 = torch.empty_like(q), torch.empty_like(q)
    ws = fb.new_kv4_workspace(2, 1, 16, HK, D, 512)
    fb.fp8bq_kv4_attention(q, cache, table, lens, y, ws)
    fb.fp8bq_kv4_attention(q, few, torch.arange(8, device="cuda", dtype=I32).view(2, 4), lens, y2, ws)
    assert torch.equal(y, y2) and bool(y.abs().sum() > 0)
    ko, vo = (torch.empty(8, HK, D, dtype=BF16, device="cuda") for _ in range(2))
    fb.fp8bq_kv4_append(q[:, :8].repeat(4, 1, 1), q[:, 8:].repeat(4, 1, 1), at * page + 5, cache)
    fb.fp8bq_kv4_read(cache, at * page + 5, ko, vo)
    want = values(*quantise(q[:, :8])).repeat(4, 1, 1)
    assert torch.equal(ko.double(), want)


def test_one_workspace_for_calls_of_any_sizes():
    ws = fb.new_kv4_workspace(40, 4, 32, 8, 256, 4096, weights=True)
    g = gen(11)
    for lens, HQ, HK, D, page in (([4000, 100], 32, 8, 128, 64), ([30] * 40, 8, 8, 64, 16),
                                  ([2000] * 3, 32, 2, 256, 32), ([4000, 100], 32, 8, 128, 64)):
        width = -(-max(lens) // page)
        cache = make_cache(g, len(lens) * width, HK, page, D)
        table = table_of(g, lens, page, width, len(lens) * width)
        lens_d = torch.tensor(lens, dtype=I32, device="cuda")
        q = rn(g, len(lens), HQ, D).to(BF16)
        y = torch.empty_like(q)
        fb.fp8bq_kv4_attention(q, cache, table, lens_d, y, ws)
        want, bound, _, _ = reference(q, cache, table, lens_d, 1, page, D ** -0.5)
        assert bool(((y.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("lens,Tq,HQ,HK", [([9000, 3], 1, 8, 2), ([5000], 4, 8, 1), ([700] * 9, 2, 16, 2)])
def test_output_in_place_of_the_queries(lens, Tq, HQ, HK):
    """y = q, with heads whose rows and tokens are split between CTAs."""
    g = gen(len(lens))
    D, page = 128, 32
    width = -(-max(lens) // page)
    cache = make_cache(g, len(lens) * width, HK, page, D)
    table = table_of(g, lens, page, width, len(lens) * width)
    lens_d = torch.tensor(lens, dtype=I32, device="cuda")
    q = rn(g, len(lens) * Tq, HQ, D).to(BF16)
    y = torch.empty_like(q)
    ws = fb.new_kv4_workspace(len(lens), Tq, HQ, HK, D, width * page)
    fb.fp8bq_kv4_attention(q, cache, table, lens_d, y, ws)
    for _ in range(3):
        own = q.clone()
        fb.fp8bq_kv4_attention(own, cache, table, lens_d, own, ws)
        assert torch.equal(own, y)


def test_empty_batches_and_tables():
    """No sequences, block tables without a column, sequences all empty: zeros, and the
    weights left as they were."""
    cache = fb.new_kv4_cache(2, 2, 16, 64)
    ws = fb.new_kv4_workspace(3, 2, 4, 2, 64, 16, weights=True)
    w = torch.full((2, 2, 16), 3.0, device="cuda")
    for B, width, n in ((0, 1, 0), (3, 0, 9), (3, 1, 0), (3, 1, -4)):
        q = torch.ones(2 * B, 4, 64, dtype=BF16, device="cuda")
        y = torch.full_like(q, 5.0)
        table = torch.zeros(B, width, dtype=I32, device="cuda")
        lens = torch.full((B,), n, dtype=I32, device="cuda")
        fb.fp8bq_kv4_attention(q, cache, table, lens, y, ws, weights=w)
        assert bool((y == 0).all()) and bool((w == 3.0).all())
    none = torch.empty(0, 2, 64, dtype=BF16, device="cuda")
    slots = torch.empty(0, dtype=I64, device="cuda")
    fb.fp8bq_kv4_append(none, none, slots, cache)
    fb.fp8bq_kv4_read(cache, slots, none, none)
    assert fb.fp8bq_poll_status(ws) == 0 and bool((cache == 0).all())


def test_streams_and_graphs():
    """The whole use of the cache on a stream of its own, captured and replayed with new
    lengths and rows; eager calls on the same workspace in between."""
    g = gen(21)
    B, HQ, HK, D, page, width = 5, 16, 2, 128, 32, 13
    cache = make_cache(g, B * width, HK, page, D)
    table = torch.randperm(B * width, generator=g, device="cuda").view(B, width).to(I32)
    lens = torch.tensor([5, 33, 200, 383, 64], dtype=I32, device="cuda")
    qkv = rn(g, B, (HQ + 2 * HK) * D).to(BF16)
    q, k, v = (qkv[:, a * D:b * D].view(B, b - a, D) for a, b in ((0, HQ), (HQ, HQ + HK),
                                                                 (HQ + HK, HQ + 2 * HK)))
    slots = torch.empty(B, dtype=I64, device="cuda")
    weights = torch.zeros(B * width, HK, page, device="cuda")
    y = torch.empty(B, HQ, D, dtype=BF16, device="cuda")
    ws = fb.new_kv4_workspace(B, 1, HQ, HK, D, width * page, weights=True)

    def place():
        at = lens.long() - 1
        slots.copy_(table.gather(1, (at // page)[:, None]).squeeze(1).long() * page + at % page)

    def step():
        fb.fp8bq_kv4_append(k, v, slots, cache, weights)
        fb.fp8bq_kv4_attention(q, cache, table, lens, y, ws, weights=weights)

    stream = torch.cuda.Stream()
    place()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        lens += 1
        place()
        qkv.copy_(rn(g, *qkv.shape))
        w0, c0 = weights.clone(), cache.clone()
        graph.replay()
        got, got_w, got_c = y.clone(), weights.clone(), cache.clone()
        want, bound, add, add_b = reference(q, cache, table, lens, 1, page, D ** -0.5)
        assert bool(((got.double() - want).abs() <= bound).all())
        weights.copy_(w0), cache.copy_(c0)
        step()
        assert torch.equal(y, got) and torch.equal(weights, got_w) and torch.equal(cache, got_c)
        # a token's weight starts again when its slot is written
        w0[slots // page, :, slots % page] = 0.0
        assert bool(((got_w.double() - w0.double() - add).abs() <=
                     add_b + (w0 + add) * 2.0 ** -23).all())
    assert fb.fp8bq_poll_status(ws) == 0


def test_shared_pages():
    """Two sequences over the same prefix pages: both add to its weights."""
    g = gen(2)
    cache = make_cache(g, 6, 2, 16, 64)
    table = torch.tensor([[0, 1, 2], [0, 1, 3]], dtype=I32, device="cuda")
    lens = torch.tensor([40, 45], dtype=I32, device="cuda")
    q = rn(g, 2, 4, 64).to(BF16)
    y = torch.empty_like(q)
    w = torch.zeros(6, 2, 16, device="cuda")
    ws = fb.new_kv4_workspace(2, 1, 4, 2, 64, 48, weights=True)
    fb.fp8bq_kv4_attention(q, cache, table, lens, y, ws, weights=w)
    want = torch.zeros(6, 2, 16, dtype=torch.float64, device="cuda")
    bounds = torch.zeros_like(want)
    for b in range(2):
        _, _, add, add_b = reference(q[b:b + 1], cache, table[b:b + 1], lens[b:b + 1], 1, 16, 0.125)
        want += add
        bounds += add_b
    assert bool(((w.double() - want).abs() <= bounds + want * 2.0 ** -22).all())
    assert float(w.sum()) == pytest.approx(8.0, rel=1e-5)


# ---------------------------------------------------------------- evict

def evict_reference(cache, table, lens, weights, new_table, budget, recent, page, D):
    cache, weights = cache.clone(), weights.clone()
    src, src_w = [p.clone() for p in parts(cache, page, D)], weights.cpu()
    dst = parts(cache, page, D)
    B, HK, pages = len(lens), cache.shape[1], cache.shape[0]
    kept = torch.full((B, HK, budget), -1, dtype=I32)
    for b in range(B):
        n = min(max(int(lens[b]), 0), table.shape[1] * page)
        row, new = table[b].tolist(), new_table[b].tolist()
        for h in range(HK):
            order = list(range(n))
            if n > budget:
                m = n - recent
                w = [float(src_w[row[i // page], h, i % page]) if 0 <= row[i // page] < pages
                     else math.nan for i in range(m)]
                best = sorted(range(m), key=lambda i: (math.isnan(w[i]), -w[i] if w[i] == w[i] else 0, i))
                order = sorted(best[:budget - recent]) + list(range(m, n))
            kept[b, h, :len(order)] = torch.tensor(order, dtype=I32)
            moves = [(row[i // page], i % page, new[j // page], j % page) for j, i in enumerate(order)]
            moves = [mv for mv in moves if 0 <= mv[0] < pages and 0 <= mv[2] < pages]
            if not moves:
                continue
            s, si, d, di = torch.tensor(moves, device="cuda").t()
            for x, y in zip(src, dst):
                y[d, h, di] = x[s, h, si]
            weights[d, h, di] = src_w.cuda()[s, h, si]
    return cache, weights, kept.cuda(), lens.clamp(0, table.shape[1] * page).clamp(max=budget)


@pytest.mark.parametrize("lens,budget,recent,HK,D,page", [
    ([100], 64, 16, 2, 128, 16), ([1, 0, 40, 41, 39, 200], 40, 7, 1, 64, 16),
    ([300, 17], 1, 0, 2, 64, 32), ([300, 17], 1, 1, 2, 64, 32), ([150, 260], 128, 128, 3, 256, 64),
    ([513, 700, 90], 130, 0, 2, 128, 128), ([1500], 1499, 700, 1, 128, 64)])
@pytest.mark.parametrize("kind", ["ties", "normal", "wild"])
def test_evict(lens, budget, recent, HK, D, page, kind):
    g = gen(sum(lens) + budget)
    B = len(lens)
    width, new_width = max(-(-n // page) for n in lens) + 1, -(-budget // page) + 1
    pages = B * (width + new_width) + 1
    guard = Guarded((pages, HK, page * 9 * D // 8), U8)
    guard.t.copy_(make_cache(g, pages, HK, page, D))
    order = torch.randperm(pages, generator=g, device="cuda").to(I32)
    table = order[:B * width].view(B, width).contiguous()
    new_table = order[B * width:B * (width + new_width)].view(B, new_width).contiguous()
    weights = rn(g, pages, HK, page)
    if kind == "ties":
        weights = (torch.rand(pages, HK, page, generator=g, device="cuda") * 4).floor()
    if kind == "wild":
        weights = weights * torch.exp2(torch.randint(-140, 120, weights.shape, generator=g, device="cuda"))
        pick = torch.randint(0, 12, weights.shape, generator=g, device="cuda")
        for i, v in enumerate((math.nan, math.inf, -math.inf, 0.0, -0.0)):
            weights[pick == i] = v
        table[0, 0] = -1
        new_table[-1, 0] = pages
    lens_d = torch.tensor(lens, dtype=I32, device="cuda")
    new_lens, kept = Guarded((B,), I32), Guarded((B, HK, budget), I32)
    want = evict_reference(guard.t, table, lens_d, weights, new_table, budget, recent, page, D)
    fb.fp8bq_kv4_evict(guard.t, table, lens_d, weights, new_table, new_lens.t, kept.t, recent, D)
    for x in (guard, new_lens, kept):
        x.check("evict")
    assert torch.equal(kept.t, want[2])
    assert torch.equal(new_lens.t, want[3])
    assert torch.equal(guard.t, want[0])
    assert torch.equal(torch.nan_to_num(weights, nan=123.0), torch.nan_to_num(want[1], nan=123.0))


def test_evict_long_sequences():
    """More tokens than the choice keeps in shared memory, and many of equal weight."""
    g = gen(4)
    page, n, budget, recent = 128, 50000, 20000, 100
    width, new_width = -(-n // page), -(-budget // page)
    pages = width + new_width
    cache = make_cache(g, pages, 1, page, 64)
    order = torch.randperm(pages, generator=g, device="cuda").to(I32)
    table, new_table = order[None, :width].contiguous(), order[None, width:].contiguous()
    weights = (torch.rand(pages, 1, page, generator=g, device="cuda") * 50).floor() / 7
    lens = torch.tensor([n], dtype=I32, device="cuda")
    new_lens, kept = torch.empty_like(lens), torch.empty(1, 1, budget, dtype=I32, device="cuda")
    t = torch.arange(n, device="cuda")
    w = weights[table[0].long()[t // page], 0, t % page]
    m = n - recent
    best = torch.sort(w[:m], descending=True, stable=True).indices[:budget - recent]
    want = torch.cat([best.sort().values, t[m:]])
    src = [p[table[0].long()[want // page], 0, want % page] for p in parts(cache, page, 64)]
    fb.fp8bq_kv4_evict(cache, table, lens, weights, new_table, new_lens, kept, recent, 64)
    assert torch.equal(kept[0, 0].long(), want) and int(new_lens) == budget
    j = torch.arange(budget, device="cuda")
    for p, s in zip(parts(cache, page, 64), src):
        assert torch.equal(p[new_table[0].long()[j // page], 0, j % page], s)
    assert torch.equal(weights[new_table[0].long()[j // page], 0, j % page], w[want])
