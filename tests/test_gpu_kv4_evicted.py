"""Attention over a cache that has been cut by weight: what is left has to be what queries
see, no more and no less, whatever the new pages held before."""
import pytest
import torch

import block_wise_fp8_gb300 as fb
from test_gpu_kv4 import (BF16, I32, evict_reference, gen, make_cache, parts, quantise,
                          reference, rn, table_of)

pytestmark = pytest.mark.gpu


def attend(q, cache, table, lens, page, weights):
    y = torch.empty_like(q)
    ws = fb.new_kv4_workspace(len(lens), 1, q.shape[1], cache.shape[1], q.shape[2],
                              table.shape[1] * page, True)
    fb.fp8bq_kv4_attention(q, cache, table, lens, y, ws, weights=weights)
    assert fb.fp8bq_poll_status(ws) == 0
    return y


def held(y, w, w0, q, cache, table, lens, page):
    """y and the weights added since w0 are those of the formula over this cache."""
    want, bound, add, add_b = reference(q, cache, table, lens, 1, page, q.shape[2] ** -0.5)
    assert bool(((y.double() - want).abs() <= bound).all())
    total = w0.double() + add
    assert bool(((w.double() - total).abs() <= add_b + total * 2.0 ** -23).all())


def evict_and_attend(g, cache, table, lens, weights, new_table, budget, recent, page, D, HQ):
    """Cuts the cache, checks it against the plain form, and twice lets a query see what is
    left: as it is, and with one more token appended."""
    B, HK = len(lens), cache.shape[1]
    want, want_w, want_kept, want_lens = evict_reference(cache, table, lens, weights, new_table,
                                                         budget, recent, page, D)
    new_lens = torch.empty(B, dtype=I32, device="cuda")
    kept = torch.empty(B, HK, budget, dtype=I32, device="cuda")
    fb.fp8bq_kv4_evict(cache, table, lens, weights, new_table, new_lens, kept, recent, D)
    assert torch.equal(kept, want_kept) and torch.equal(new_lens, want_lens)
    assert torch.equal(cache, want) and torch.equal(weights, want_w)
    q = rn(g, B, HQ, D).to(BF16)
    y = attend(q, cache, new_table, new_lens, page, weights)
    held(y, weights, want_w, q, want, new_table, want_lens, page)
    k, v = rn(g, B, HK, D).to(BF16), rn(g, B, HK, D).to(BF16)
    at = new_lens.long()
    pg = new_table.long().gather(1, (at // page)[:, None])[:, 0]
    slots = torch.where(pg >= 0, pg * page + at % page, -1)
    fb.fp8bq_kv4_append(k, v, slots, cache, weights)
    p4, on = parts(want, page, D), slots >= 0
    for i, x in ((0, k), (2, v)):
        p4[i][pg[on], :, at[on] % page], p4[i + 1][pg[on], :, at[on] % page] = quantise(x[on])
    w0 = weights.clone()
    assert bool((w0[pg[on], :, at[on] % page] == 0).all())
    y = attend(q, cache, new_table, new_lens + 1, page, weights)
    held(y, weights, w0, q, want, new_table, want_lens + 1, page)


def setup(g, lens, budget, HQ, HK, D, page):
    """A cache whose free pages hold NaN scales, tables with -1 behind the sequences' ends and
    the weights of one attention."""
    B, width, new_width = len(lens), max(1, max(-(-n // page) for n in lens)), budget // page + 1
    pages = B * (width + new_width) + 1
    cache = make_cache(g, pages, HK, page, D)
    table = table_of(g, lens, page, width, pages)
    free = torch.ones(pages, dtype=torch.bool, device="cuda")
    free[table[table >= 0].long()] = False
    cache[free] = 0xFF
    new_table = free.nonzero()[:B * new_width, 0].view(B, new_width).to(I32)
    lens = torch.tensor(lens, dtype=I32, device="cuda")
    weights = torch.zeros(pages, HK, page, device="cuda")
    attend(rn(g, B, HQ, D).to(BF16), cache, table, lens, page, weights)
    return cache, table, lens, weights, new_table


@pytest.mark.parametrize("lens,budget,recent,HQ,HK,D,page", [
    ([100, 64, 65, 0, 1], 64, 16, 8, 2, 128, 16), ([300, 17, 2000], 40, 0, 3, 3, 64, 32),
    ([900, 128, 700], 256, 256, 16, 2, 256, 64), ([3000, 1500], 1000, 100, 8, 1, 128, 128)])
def test_queries_see_what_is_kept(lens, budget, recent, HQ, HK, D, page):
    g = gen(budget)
    evict_and_attend(g, *setup(g, lens, budget, HQ, HK, D, page), budget, recent, page, D, HQ)


def without_holes(table, lens, page, pages):
    """The tables without the pages that are not there, and the lengths without their
    tokens."""
    t = torch.arange(table.shape[1], device="cuda")
    here = (table >= 0) & (table < pages)
    tokens = (lens[:, None] - t * page).clamp(0, page) * here
    order = torch.argsort((~here).long(), dim=1, stable=True)
    return (torch.where(here, table, -1).gather(1, order).contiguous(),
            tokens.sum(1).to(I32))


@pytest.mark.parametrize("HQ,HK,D,page", [(8, 2, 128, 16), (3, 1, 64, 32), (4, 4, 256, 16)])
def test_pages_that_are_not_there_are_left_out_first(HQ, HK, D, page):
    """Pages missing among the heavy tokens, among the recent ones (the last, partly filled
    page too), in sequences within the budget, and all of a sequence's."""
    g = gen(D + page)
    budget, recent = 6 * page + 3, 2 * page
    lens = [20 * page + 5, 9 * page, 20 * page + 5, 4 * page + 1, 3 * page, 2 * page]
    cache, table, lens, weights, new_table = setup(g, lens, budget, HQ, HK, D, page)
    pages = cache.shape[0]
    table[0, 3] = table[0, 7] = -1           # heavy
    table[1, 7], table[1, 8] = pages, -5     # recent
    table[2, 20] = -1                        # recent, the last one
    table[3, 1] = 2 ** 31 - 1                # within the budget
    table[5] = -1                            # all
    packed, short = without_holes(table, lens, page, pages)
    assert short.tolist() == [18 * page + 5, 7 * page, 20 * page, 3 * page + 1, 3 * page, 0]
    # no query can tell the two tables apart
    q = rn(g, len(lens), HQ, D).to(BF16)
    for tb, n in ((table, lens), (packed, short)):
        w = torch.zeros_like(weights)
        held(attend(q, cache, tb, n, page, w), w, torch.zeros_like(w), q, cache, table, lens, page)
    evict_and_attend(g, cache, packed, short, weights, new_table, budget, recent, page, D, HQ)


def test_new_pages_that_are_not_there():
    """Tokens that are kept without a place are seen by no query."""
    g = gen(9)
    budget, recent, HQ, HK, D, page = 70, 20, 8, 2, 128, 16
    cache, table, lens, weights, new_table = setup(g, [300, 40, 90], budget, HQ, HK, D, page)
    new_table[0, 1], new_table[1, 0], new_table[2, 4] = -1, cache.shape[0], -9
    new_table[new_table >= cache.shape[0]] = -1
    evict_and_attend(g, cache, table, lens, weights, new_table, budget, recent, page, D, HQ)
