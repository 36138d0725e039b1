"""Attention of a served decoder layer and its cache in 4 bits, as cases to be timed.

Five operators between the query/key norm and the output projection:

  prompt    causal attention over whole prompts: packed sequences of different
            lengths, grouped heads, BF16 in and out
  append    rows of keys and values written into a paged cache as E2M1 codes with
            one E4M3 scale for 16 values, and read back as BF16 (the operator that
            reads them is what a prompt over a cached prefix starts with)
  attend    attention of one or a few new tokens of every request over its pages;
            with `weights` the softmax weight that each cached token receives is
            added up for every key/value head
  evict     the tokens with the largest weights, and the last ones, of every
            sequence and key/value head, moved to pages of their own

A page holds, for every key/value head, its tokens' key codes, key scales, value
codes and value scales, one after the other; the code of a row's value 2i is the
low half of its byte i.

`run` computes a case in elementary torch operations, or, where `own` is true,
by the calls a user of block_wise_fp8_gb300 makes; `exact` computes it in 64
bits from the definitions.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TIES = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a few short requests, down to one token, the sizes of this repository's example layer
        dict(name="prompt_short", op="prompt", S=7, T=301, HQ=16, HK=2, D=128),
        # a ragged prefill batch, the heads of this repository's norm-and-rotation cases
        dict(name="prompt_ragged", op="prompt", S=9, T=4099, HQ=64, HK=8, D=128),
        # heads of 64 in groups of three
        dict(name="prompt_d64", op="prompt", S=3, T=2039, HQ=12, HK=4, D=64),
        # one long prompt
        dict(name="prompt_long", op="prompt", S=1, T=16384, HQ=32, HK=4, D=128),
        # the rows of a decode batch, and of a long prefill
        dict(name="append_m64", op="append", T=64, HK=8, D=128, page=64),
        dict(name="append_t8192", op="append", T=8192, HK=8, D=128, page=64),
        # one request's next token over a short context: latency
        dict(name="attend_m1", op="attend", B=1, Tq=1, HQ=64, HK=8, D=128, page=64, longest=701,
             weights=False),
        # a decode batch of requests of all lengths
        dict(name="attend_m64", op="attend", B=64, Tq=1, HQ=64, HK=8, D=128, page=64,
             longest=8192, weights=False),
        # few requests with very long contexts
        dict(name="attend_long", op="attend", B=8, Tq=1, HQ=64, HK=8, D=128, page=128,
             longest=131072, weights=False),
        # four tokens a request (drafted ones among them), small pages, weights added up
        dict(name="attend_draft", op="attend", B=16, Tq=4, HQ=32, HK=8, D=128, page=16,
             longest=16384, weights=True),
        # one request some tokens over its budget, and a batch cut to a quarter
        dict(name="evict_b1", op="evict", B=1, HK=8, D=128, page=64, longest=2203, budget=2048,
             recent=256),
        dict(name="evict_b32", op="evict", B=32, HK=8, D=128, page=64, longest=16384, budget=4096,
             recent=512),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "append", "attend", "attend", "attend", "evict"])
    D = rng.choice([64, 128])
    if op == "prompt":
        T, HK, G = _spread(rng, 1, 8192), _spread(rng, 1, 8), rng.randint(1, 8)
        return dict(op="prompt", S=min(T, _spread(rng, 1, 24)), T=T, HQ=HK * G, HK=HK,
                    D=rng.choice([64, 80, 96, 128]))
    HK, page = _spread(rng, 1, 8), rng.choice([16, 32, 64, 128])
    if op == "append":
        return dict(op="append", T=_spread(rng, 1, 8192), HK=HK, D=D, page=page)
    B = _spread(rng, 1, 64)
    if op == "attend":
        return dict(op="attend", B=B, Tq=rng.choice([1, 1, 2, 5]), HQ=HK * rng.randint(1, 16),
                    HK=HK, D=D, page=page, longest=_spread(rng, 1, 65536 // max(1, B // 4)),
                    weights=rng.random() < 0.4)
    longest = _spread(rng, 64, 16384 if B <= 32 else 8192)
    budget = _spread(rng, 16, longest)
    return dict(op="evict", B=B, HK=HK, D=D, page=page, longest=longest, budget=budget,
                recent=rng.randint(0, budget // 2))


# ---------------------------------------------------------------- inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _lengths(g, n, total):
    """n lengths of at least one that add up to total, most of it with a few."""
    w = torch.rand(n, generator=g, device="cuda") ** 2 + 0.01
    left = total - n
    cuts = (w.cumsum(0) / w.sum() * left).round().long()
    cuts[-1] = left
    return torch.diff(cuts, prepend=cuts.new_zeros(1)) + 1


def _heads(g, T, HQ, HK, D):
    """Slices of packed QKV rows: normed and rotated queries and keys, values."""
    qkv = _randn(g, T, (HQ + 2 * HK) * D).to(torch.bfloat16)
    return (qkv[:, :HQ * D].view(T, HQ, D), qkv[:, HQ * D:(HQ + HK) * D].view(T, HK, D),
            qkv[:, (HQ + HK) * D:].view(T, HK, D))


def _page_parts(cache, page, D):
    """Key codes, key scales, value codes and value scales of [..., page bytes]."""
    c, s = page * D // 2, page * D // 16
    parts = cache.split([c, s, c, s], -1)
    return [p.unflatten(-1, (page, -1)) for p in parts]


def _cache(g, pages, HK, D, page):
    """A cache of normal keys and values as group-16 quantisation leaves them."""
    cache = torch.empty(pages, HK, page * 9 * D // 8, dtype=torch.uint8, device="cuda")
    ties = torch.tensor(TIES, device="cuda")
    for p0 in range(0, pages, 512):
        part = cache[p0:p0 + 512]
        for i, (codes, scales) in enumerate(zip(*[iter(_page_parts(part, page, D))] * 2)):
            v = _randn(g, *codes.shape[:-1], D) * 2.2
            code = torch.bucketize(v.abs(), ties, out_int32=True).to(torch.uint8)
            code = code | (v < 0).to(torch.uint8) * 8
            codes.copy_(code[..., 0::2] | code[..., 1::2] * 16)
            s = torch.rand(scales.shape, generator=g, device="cuda") * 0.5 + 0.25
            scales.copy_(s.to(torch.float8_e4m3fn).view(torch.uint8))
    return cache


def _tables(g, lens, page, longest, pages):
    """Block tables [B, pages of the longest] with pages in random order."""
    need = -(-lens // page)
    width = -(-longest // page)
    order = torch.randperm(pages, generator=g, device="cuda")
    first = need.cumsum(0) - need
    col = torch.arange(width, device="cuda")[None, :]
    at = (first[:, None] + col).clamp(max=pages - 1)
    return torch.where(col < need[:, None], order[at], -1).to(torch.int32), order[int(need.sum()):]


def _ragged(g, B, longest):
    """Lengths of a batch: one the longest, the others anything below, even over the logarithm."""
    u = torch.rand(B, generator=g, device="cuda")
    lens = torch.exp(math.log(max(1.0, longest / 16)) * (1 - u) + math.log(longest) * u)
    lens = lens.long().clamp(1, longest)
    lens[int(torch.randint(0, B, (1,), generator=g, device="cuda"))] = longest
    return lens


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    s = {"case": case}
    op, D, HK = case["op"], case["D"], case["HK"]
    if op == "prompt":
        T, HQ = case["T"], case["HQ"]
        s["q"], s["k"], s["v"] = _heads(g, T, HQ, HK, D)
        lens = _lengths(g, case["S"], T)
        s["offsets"] = torch.cat([lens.new_zeros(1), lens.cumsum(0)]).to(torch.int32)
        s["y"] = torch.empty(T, HQ, D, dtype=torch.bfloat16, device="cuda")
        return s
    page = case["page"]
    if op == "append":
        T = case["T"]
        _, s["k"], s["v"] = _heads(g, T, HK, HK, D)
        pages = 2 * -(-T // page)
        s["cache"] = torch.zeros(pages, HK, page * 9 * D // 8, dtype=torch.uint8, device="cuda")
        s["slots"] = torch.randperm(pages * page, generator=g, device="cuda")[:T]
        s["k_out"] = torch.empty(T, HK, D, dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.empty(T, HK, D, dtype=torch.bfloat16, device="cuda")
        return s
    B, longest = case["B"], case["longest"]
    lens = _ragged(g, B, longest)
    s["lens"] = lens.to(torch.int32)
    if op == "attend":
        HQ, Tq = case["HQ"], case["Tq"]
        pages = B * -(-longest // page) + 3
        s["q"] = _heads(g, B * Tq, HQ, HK, D)[0]
        s["cache"] = _cache(g, pages, HK, D, page)
        s["table"], _ = _tables(g, lens, page, longest, pages)
        s["y"] = torch.empty(B * Tq, HQ, D, dtype=torch.bfloat16, device="cuda")
        s["weights"] = None
        if case["weights"]:
            s["weights"] = torch.rand(pages, HK, page, generator=g, device="cuda")
        return s
    budget = case["budget"]
    width = -(-budget // page)
    pages = B * (-(-longest // page) + width)
    s["cache"] = _cache(g, pages, HK, D, page)
    s["table"], rest = _tables(g, lens, page, longest, pages)
    s["new_table"] = rest[:B * width].view(B, width).to(torch.int32)
    # a few tokens draw most of the weight; many of the small ones are equal
    w = torch.rand(pages, HK, page, generator=g, device="cuda") ** 8
    s["weights"] = (w * 4096).round() / 4096
    s["kept"] = torch.empty(B, HK, budget, dtype=torch.int32, device="cuda")
    s["new_lens"] = torch.empty(B, dtype=torch.int32, device="cuda")
    col = torch.arange(width * page, device="cuda")
    slots = s["new_table"].long()[:, col // page] * page + col % page
    live = col[None, :] < lens.clamp(max=budget)[:, None]
    s["slots"] = torch.where(live, slots, -1)[:, :budget].reshape(-1).contiguous()
    s["k_out"] = torch.zeros(B * budget, HK, D, dtype=torch.bfloat16, device="cuda")
    s["v_out"] = torch.zeros(B * budget, HK, D, dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_prompt(s):
    import block_wise_fp8_gb300 as fb
    if "ws" not in s:
        s["ws"] = fb.new_workspace(fb.OP_PROMPT_ATTENTION, s["case"]["T"], s["case"]["HQ"],
                                   s["case"]["D"])
    fb.fp8bq_prompt_attention(s["q"], s["k"], s["v"], s["offsets"], s["y"], s["ws"])
    return s["y"]


def _own_append(s):
    import block_wise_fp8_gb300 as fb
    fb.fp8bq_kv4_append(s["k"], s["v"], s["slots"], s["cache"])
    fb.fp8bq_kv4_read(s["cache"], s["slots"], s["k_out"], s["v_out"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _own_attend(s):
    import block_wise_fp8_gb300 as fb
    c = s["case"]
    if "ws" not in s:
        s["ws"] = fb.new_kv4_workspace(c["B"], c["Tq"], c["HQ"], c["HK"], c["D"],
                                       s["table"].shape[1] * c["page"], weights=c["weights"])
    fb.fp8bq_kv4_attention(s["q"], s["cache"], s["table"], s["lens"], s["y"], s["ws"],
                           weights=s["weights"])
    return {"y": s["y"], "weights": s["weights"]}


def _own_evict(s):
    import block_wise_fp8_gb300 as fb
    c = s["case"]
    fb.fp8bq_kv4_evict(s["cache"], s["table"], s["lens"], s["weights"], s["new_table"],
                       s["new_lens"], s["kept"], c["recent"], c["D"])
    fb.fp8bq_kv4_read(s["cache"], s["slots"], s["k_out"], s["v_out"])
    return {"kept": s["kept"], "lens": s["new_lens"], "k": s["k_out"], "v": s["v_out"],
            "weights": _weights_of(s)}


def _weights_of(s):
    """The moved weights: those of the pages that the new table names."""
    return s["weights"][s["new_table"]]


def _plain_prompt(s):
    c = s["case"]
    T, HQ, HK, D = c["T"], c["HQ"], c["HK"], c["D"]
    tok = torch.arange(T, device="cuda")
    seq = torch.bucketize(tok, s["offsets"][1:], right=True)
    k = s["k"].float().permute(1, 2, 0)
    v = s["v"].float().transpose(0, 1)
    y = torch.empty(T, HQ, D, dtype=torch.bfloat16, device="cuda")
    for t0 in range(0, T, 512):  # scores of 512 tokens at a time fit the memory
        t1 = min(T, t0 + 512)
        q = s["q"][t0:t1].float().view(t1 - t0, HK, HQ // HK, D).permute(1, 2, 0, 3)
        p = torch.matmul(q.flatten(1, 2), k[:, :, :t1]) * D ** -0.5
        p = p.view(HK, HQ // HK, t1 - t0, t1)
        seen = (seq[t0:t1, None] == seq[None, :t1]) & (tok[t0:t1, None] >= tok[None, :t1])
        p = p.masked_fill_(~seen, -math.inf)
        p = torch.exp(p.sub_(p.amax(-1, keepdim=True)))
        o = torch.matmul(p.flatten(1, 2), v[:, :t1]).view(HK, HQ // HK, t1 - t0, D)
        o = o / p.sum(-1, keepdim=True)
        y[t0:t1] = o.permute(2, 0, 1, 3).reshape(t1 - t0, HQ, D).to(torch.bfloat16)
    return y


def _values(codes, scales):
    """What codes [..., D/2] and scales [..., D/16] stand for, in 32 bits."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    v = torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], -1).flatten(-2)
    s = scales.contiguous().view(torch.float8_e4m3fn).float()
    return v * s.repeat_interleave(16, -1)


def _plain_append(s):
    c = s["case"]
    page, D = c["page"], c["D"]
    slots, ties = s["slots"], torch.tensor(TIES, device="cuda")
    out = []
    parts = _page_parts(s["cache"], page, D)
    for rows, codes, scales in ((s["k"], parts[0], parts[1]), (s["v"], parts[2], parts[3])):
        x = rows.float().unflatten(-1, (D // 16, 16))
        sc = (x.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn).float()
        sc = sc.clamp(min=2.0 ** -9)
        r = x / sc[..., None]
        # nearest, ties to the even code: up from the odd codes' upper ties alone
        a = r.abs()
        code = torch.bucketize(a, ties, out_int32=True)
        tie = (a == ties[code.clamp(max=6)]) & (code % 2 == 1)
        code = (code + tie.int()).to(torch.uint8) | (torch.signbit(r)).to(torch.uint8) * 8
        code = code.flatten(-2)
        codes[slots // page, :, slots % page] = code[..., 0::2] | code[..., 1::2] * 16
        scales[slots // page, :, slots % page] = sc.to(torch.float8_e4m3fn).view(torch.uint8)
        out.append(_values(codes[slots // page, :, slots % page],
                           scales[slots // page, :, slots % page]).to(torch.bfloat16))
    return {"k": out[0], "v": out[1]}


def _plain_attend(s):
    c = s["case"]
    B, Tq, HQ, HK, D, page = c["B"], c["Tq"], c["HQ"], c["HK"], c["D"], c["page"]
    table = s["table"].long().clamp(min=0)
    n = table.shape[1] * page
    parts = _page_parts(s["cache"][table], page, D)  # [B, pages, HK, page, ...]
    k = _values(parts[0], parts[1]).transpose(1, 2).reshape(B, HK, n, D)
    q = s["q"].float().view(B, Tq, HK, HQ // HK, D).permute(0, 2, 3, 1, 4)
    p = torch.matmul(q.flatten(2, 3), k.transpose(2, 3)) * D ** -0.5
    p = p.view(B, HK, HQ // HK, Tq, n)
    ends = s["lens"][:, None] - (Tq - 1) + torch.arange(Tq, device="cuda")[None, :]
    seen = torch.arange(n, device="cuda")[None, None, :] < ends[:, :, None]
    p = p.masked_fill_(~seen[:, None, None], -math.inf)
    p = torch.exp(p - p.amax(-1, keepdim=True).clamp(min=-1e30))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    v = _values(parts[2], parts[3]).transpose(1, 2).reshape(B, HK, n, D)
    o = torch.matmul(p.flatten(2, 3), v).view(B, HK, HQ // HK, Tq, D)
    y = o.permute(0, 3, 1, 2, 4).reshape(B * Tq, HQ, D).to(torch.bfloat16)
    if s["weights"] is not None:
        add = p.sum((2, 3)).view(B, HK, n // page, page).transpose(1, 2)
        live = s["table"] >= 0
        s["weights"][s["table"][live].long()] += add[live]
    return {"y": y, "weights": s["weights"]}


def _rows_of(x, table, page):
    """[pages, HK, page, ...] as [B, HK, tokens, ...] by a block table."""
    return x[table.long().clamp(min=0)].transpose(1, 2).flatten(2, 3)


def _plain_evict(s):
    c = s["case"]
    B, HK, D, page, budget = c["B"], c["HK"], c["D"], c["page"], c["budget"]
    lens = s["lens"].long()
    w = _rows_of(s["weights"], s["table"], page)
    n = w.shape[2]
    pos = torch.arange(n, device="cuda")
    live = pos[None, :] < lens[:, None]
    late = live & (pos[None, :] >= (lens - c["recent"])[:, None])
    key = torch.where(late[:, None], math.inf, torch.where(live[:, None], w, -1.0))
    take = min(budget, n)
    top = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :take]
    some = torch.arange(take, device="cuda")[None, :] < lens.clamp(max=budget)[:, None]
    top = torch.where(some[:, None], top, n).sort(-1).values
    got = top < n
    kept = torch.full((B, HK, budget), -1, dtype=torch.int32, device="cuda")
    kept[..., :take] = torch.where(got, top, -1).to(torch.int32)
    at = top.clamp(max=n - 1)
    parts = _page_parts(s["cache"], page, D)
    b, h, i = got.nonzero(as_tuple=True)
    to = s["new_table"].long()[b, i // page]
    outs = []
    for codes, scales in ((parts[0], parts[1]), (parts[2], parts[3])):
        moved = [_rows_of(x, s["table"], page).gather(2, at[..., None].expand(
            -1, -1, -1, x.shape[-1])) for x in (codes, scales)]
        v = torch.zeros(B, HK, budget, D, dtype=torch.bfloat16, device="cuda")
        v[:, :, :take] = torch.where(got[..., None], _values(*moved), 0.0).to(torch.bfloat16)
        outs.append(v.transpose(1, 2).reshape(B * budget, HK, D))
        for x, m in zip((codes, scales), moved):
            x[to, h, i % page] = m[b, h, i]
    s["weights"][to, h, i % page] = w.gather(2, at)[b, h, i]
    return {"kept": kept, "lens": lens.clamp(max=budget).to(torch.int32), "k": outs[0],
            "v": outs[1], "weights": _weights_of(s)}


_OWN = {"prompt": _own_prompt, "append": _own_append, "attend": _own_attend, "evict": _own_evict}
_PLAIN = {"prompt": _plain_prompt, "append": _plain_append, "attend": _plain_attend,
          "evict": _plain_evict}


# ---------------------------------------------------------------- work

def work(case):
    D, HK = case["D"], case["HK"]
    row = 9 * D // 8  # bytes of a token's key and value in a page
    if case["op"] == "prompt":
        T, HQ, S = case["T"], case["HQ"], case["S"]
        # pairs of a query and a key: lengths that share T as _lengths deals them
        w = sum((i / S) ** 4 for i in range(1, S + 1)) / sum((i / S) ** 2 for i in range(1, S + 1)) ** 2
        pairs = T * T * w / 2 + T / 2
        return {"bytes": int(4 * T * (HQ + HK) * D), "flops": int(4 * pairs * HQ * D)}
    if case["op"] == "append":
        n = case["T"] * HK
        return {"bytes": int(n * (8 * D + 2 * row) + 8 * case["T"]), "flops": 0}
    mean = case["longest"] * (1 - 1 / 16) / math.log(16)  # of _ragged's lengths
    tokens = case["longest"] + (case["B"] - 1) * max(1.0, mean)
    if case["op"] == "attend":
        rows = case["B"] * case["Tq"] * case["HQ"]
        return {"bytes": int(tokens * HK * (row + (8 if case["weights"] else 0)) + 4 * rows * D),
                "flops": int(4 * tokens * case["HQ"] * case["Tq"] * D)}
    kept = min(case["budget"], case["longest"]) + (case["B"] - 1) * min(case["budget"], mean)
    return {"bytes": int(HK * (4 * tokens + kept * (3 * row + 4 + 4 + 4 + 4 * D))), "flops": 0}


# ---------------------------------------------------------------- 64 bits

def _decode(codes, scales):
    """Values of codes [n, D/2] and scales [n, D/16] from the formats' fields."""
    nib = torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1).double()
    sign, mag = torch.where(nib >= 8, -1.0, 1.0).double(), nib % 8
    e, m = torch.floor(mag / 2), mag % 2
    v = sign * torch.where(e > 0, (1 + m / 2) * torch.exp2(e - 1), m / 2)
    b = scales.double()
    e, m = torch.floor(b / 8) % 16, b % 8
    s = torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m / 8 * 2.0 ** -6)
    return (v.view(codes.shape[0], -1, 16) * s[:, :, None]).reshape(codes.shape[0], -1)


def _token_bytes(s, b, h):
    """Codes and scales of every cached token of one sequence and head."""
    c = s["case"]
    page, D, n = c["page"], c["D"], int(s["lens"][b])
    t = torch.arange(n, device="cuda")
    blk = s["cache"][s["table"][b].long()[t // page], h]  # [n, page bytes]
    i = (t % page)[:, None]
    out, start = [], 0
    for width in (D // 2, D // 16, D // 2, D // 16):
        cols = start + i * width + torch.arange(width, device="cuda")[None, :]
        out.append(blk.gather(1, cols))
        start += page * width
    return out


def _nearest(x, grid):
    """Value of `grid` (ascending) nearest to each x, ties to the even place."""
    grid = torch.tensor(grid, dtype=torch.float64, device="cuda")
    lo = (torch.bucketize(x, grid, right=True) - 1).clamp(0, len(grid) - 2)
    down, up = x - grid[lo], grid[lo + 1] - x
    take = torch.where(down == up, lo % 2 == 1, down > up)
    return grid[lo + take.long()]


def exact(case, seed):
    s = prepare(case, seed)
    D, HK = case["D"], case["HK"]
    if case["op"] == "prompt":
        G = case["HQ"] // HK
        y = torch.empty(case["T"], case["HQ"], D, dtype=torch.float64, device="cuda")
        ends = s["offsets"].tolist()
        for a, b in zip(ends, ends[1:]):
            for h in range(case["HQ"]):
                q, k, v = (x[a:b, i].double() for x, i in ((s["q"], h), (s["k"], h // G),
                                                         (s["v"], h // G)))
                for r in range(0, b - a, 2048):
                    e = min(b - a, r + 2048)
                    p = q[r:e] @ k[:e].t() / math.sqrt(D)
                    p[:, r:].masked_fill_(torch.ones_like(p[:, r:]).triu(1).bool(), -math.inf)
                    y[a + r:a + e, h] = torch.softmax(p, -1) @ v[:e]
        return y
    if case["op"] == "append":
        grid = [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)]
        scale_grid = [m * 2.0 ** -9 for m in range(8)] + grid[:-1]
        out = {}
        for n in ("k", "v"):
            x = s[n].double().reshape(-1, 16)
            sc = _nearest((x.abs().amax(1) / 6).clamp(max=448.0), scale_grid).clamp(min=2.0 ** -9)
            v = _nearest((x.abs() / sc[:, None]).clamp(max=6.0), list(E2M1))
            out[n] = (torch.sign(x) * v * sc[:, None]).view(s[n].shape)
        return out
    if case["op"] == "attend":
        B, Tq, HQ = case["B"], case["Tq"], case["HQ"]
        G = HQ // HK
        y = torch.zeros(B, Tq, HQ, D, dtype=torch.float64, device="cuda")
        w = None if s["weights"] is None else s["weights"].double()
        q = s["q"].double().view(B, Tq, HQ, D)
        for b in range(B):
            n = int(s["lens"][b])
            t = torch.arange(n, device="cuda")
            for h in range(HK):
                kc, ks, vc, vs = _token_bytes(s, b, h)
                k, v = _decode(kc, ks), _decode(vc, vs)
                for i in range(Tq):
                    m = n - (Tq - 1 - i)
                    if m <= 0:
                        continue
                    p = torch.softmax(q[b, i, h * G:(h + 1) * G] @ k[:m].t() / math.sqrt(D), -1)
                    y[b, i, h * G:(h + 1) * G] = p @ v[:m]
                    if w is not None:
                        blk = s["table"][b].long()[t[:m] // case["page"]]
                        w[blk, h, t[:m] % case["page"]] += p.sum(0)
        return {"y": y.view(B * Tq, HQ, D), "weights": w}
    # what is kept is whole numbers and copies: one sequence and head at a time
    B, budget, page = case["B"], case["budget"], case["page"]
    k_out = torch.zeros(B, budget, HK, D, dtype=torch.float64, device="cuda")
    v_out = torch.zeros_like(k_out)
    moved = s["weights"].double().clone()
    for b in range(B):
        n = int(s["lens"][b])
        t = torch.arange(n, device="cuda")
        old = min(n, max(0, n - case["recent"]))
        for h in range(HK):
            w = s["weights"][s["table"][b].long()[t // page], h, t % page].double()
            keep = t
            if n > budget:
                best = torch.argsort(-w[:old], stable=True)[:budget - (n - old)]
                keep = torch.cat([best, t[old:]]).sort().values
            kc, ks, vc, vs = _token_bytes(s, b, h)
            k_out[b, :len(keep), h] = _decode(kc[keep], ks[keep])
            v_out[b, :len(keep), h] = _decode(vc[keep], vs[keep])
            to = torch.arange(len(keep), device="cuda")
            moved[s["new_table"][b].long()[to // page], h, to % page] = w[keep]
    return {"kept": None, "lens": None, "k": k_out.view(B * budget, HK, D),
            "v": v_out.view(B * budget, HK, D), "weights": moved[s["new_table"]]}
