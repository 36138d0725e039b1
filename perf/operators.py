"""The operators beside the block-FP8 linears, as cases to be timed.

Four operators of a served decoder layer:

  moe    a whole mixture-of-experts layer for up to 64 tokens over block-FP8
         experts: top-k routing from the router's logits, group-128 activation
         quantisation, gate and up products, SiLU(gate) * up, quantisation of
         the hidden rows, down product, weighted sum over the token's experts
  lora   low-rank adapters of many requests beside a shared projection:
         y = base + scale[a] * B[a] (A[a] x) with each token's own adapter a
  group  token indices sorted by adapter, with one segment per adapter
  rope   RMSNorm of each query and key head and the rotary embedding, one pass
         over the slices of a packed QKV projection

`run` computes a case in elementary torch operations, or, where `own` is true,
by the calls a user of block_wise_fp8_gb300 makes; `exact` computes it in 64
bits from the definitions.
"""
import math

import torch

own = False

E4M3_MAX = 448.0


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token through a small expert layer: launch and dependency latency
        dict(name="moe_m1_small", op="moe", M=1, E=64, H=2048, I=768, topk=4, score="softmax",
             renorm=True, scale=1.0, bias=False),
        # one decoded token, the expert sizes of this repository's grouped GEMM
        dict(name="moe_m1", op="moe", M=1, E=32, H=7168, I=2048, topk=8, score="sigmoid",
             renorm=True, scale=2.5, bias=True),
        # a small decode batch that reaches nearly every expert of the same layer
        dict(name="moe_m16", op="moe", M=16, E=32, H=7168, I=2048, topk=8, score="sigmoid",
             renorm=True, scale=2.5, bias=True),
        # an odd decode batch over many experts, two tokens in most of them or more
        dict(name="moe_m61", op="moe", M=61, E=128, H=4096, I=1408, topk=8, score="softmax",
             renorm=False, scale=1.0, bias=False),
        # one decoded token with its adapter
        dict(name="lora_m1", op="lora", M=1, L=4, R=16, K=6144, N=6144, ranks="full", runs=1),
        # a decode batch of many requests, adapters of mixed rank in no order
        dict(name="lora_m64", op="lora", M=64, L=32, R=32, K=6144, N=6144, ranks="mixed", runs=1),
        # a ragged prefill of a few requests into a wide projection
        dict(name="lora_m2039", op="lora", M=2039, L=8, R=64, K=4096, N=14336, ranks="mixed",
             runs=127),
        # a full prefill batch into the up projection of this repository's benchmark
        dict(name="lora_m4096", op="lora", M=4096, L=4, R=64, K=6144, N=24576, ranks="full",
             runs=512),
        # grouping of a decode batch, and of a long prefill batch
        dict(name="group_m64", op="group", M=64, L=32, runs=1),
        dict(name="group_m16384", op="group", M=16384, L=128, runs=61),
        # one decoded token: latency alone
        dict(name="rope_t1", op="rope", T=1, HQ=64, HK=8, D=128, rot=128, inter=False, P=32768),
        # a long prefill
        dict(name="rope_t8192", op="rope", T=8192, HQ=64, HK=8, D=128, rot=128, inter=False,
             P=32768),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["moe", "moe", "lora", "lora", "group", "rope"])
    if op == "moe":
        H, I = 16 * _spread(rng, 32, 448), 128 * _spread(rng, 2, 16)
        E = min(_spread(rng, 8, 128), 128 * 4096 * 1408 // (H * I))
        score = rng.choice(["softmax", "sigmoid"])
        return dict(op="moe", M=_spread(rng, 1, 64), E=E, H=H, I=I,
                    topk=rng.randint(1, min(8, E)), score=score, renorm=rng.random() < 0.5,
                    scale=rng.choice([1.0, 2.5]), bias=score == "sigmoid" and rng.random() < 0.5)
    if op == "lora":
        M, K, N = _spread(rng, 1, 4096), 16 * _spread(rng, 32, 448), 8 * _spread(rng, 64, 2048)
        return dict(op="lora", M=M, L=_spread(rng, 1, 64), R=8 * rng.randint(1, 8), K=K, N=N,
                    ranks=rng.choice(["full", "mixed"]), runs=_spread(rng, 1, 512))
    if op == "group":
        return dict(op="group", M=_spread(rng, 1, 16384), L=_spread(rng, 1, 256),
                    runs=_spread(rng, 1, 512))
    D = 16 * rng.randint(4, 12)
    return dict(op="rope", T=_spread(rng, 1, 4096), HQ=_spread(rng, 1, 64), HK=_spread(rng, 1, 8),
                D=D, rot=rng.choice([D, 64]), inter=rng.random() < 0.5,
                P=_spread(rng, 4096, 131072))


# ---------------------------------------------------------------- inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _experts(g, E, rows, cols):
    """E4M3 codes [E, rows, cols] of normal weights, as absmax block quantisation
    leaves them, and FP32 128 x 128 block scales."""
    q = torch.empty(E, rows, cols, dtype=torch.float8_e4m3fn, device="cuda")
    for e in range(E):
        q[e] = (_randn(g, rows, cols) * 112.0).clamp_(-E4M3_MAX, E4M3_MAX)
    s = torch.rand(E, -(-rows // 128), -(-cols // 128), generator=g, device="cuda")
    return q, (s * 0.4 + 0.8) * (0.02 / 112.0)


def _adapter_ids(g, M, L, runs):
    """Adapter of each token in runs of neighbours, -1 for a few: every adapter
    is met where there are runs enough."""
    n = -(-M // runs)
    ids = torch.randperm(max(n, L + 1), generator=g, device="cuda")[:n] % (L + 1)
    ids = torch.where(ids == L, -1 if n > 1 else 0, ids)
    return ids.repeat_interleave(runs)[:M].to(torch.int32).contiguous()


def _ranks(case):
    R = case["R"]
    full = case["ranks"] == "full"
    return [R if full else max(1, R >> (a % 3)) for a in range(case["L"])]


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "moe":
        M, E, H, I = case["M"], case["E"], case["H"], case["I"]
        x = _randn(g, M, H)
        big = torch.rand(H, generator=g, device="cuda") < 0.01
        s["x"] = (x * torch.where(big, 10.0, 1.0)).to(torch.bfloat16)
        s["logits"] = _randn(g, M, E) * 1.5
        s["bias"] = _randn(g, E) * 0.1 if case["bias"] else None
        s["w13"], s["s13"] = _experts(g, E, 2 * I, H)
        s["w2"], s["s2"] = _experts(g, E, H, I)
        s["y"] = torch.empty(M, H, dtype=torch.bfloat16, device="cuda")
        s["ids"] = torch.empty(M, case["topk"], dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty(M, case["topk"], dtype=torch.float32, device="cuda")
    elif case["op"] in ("lora", "group"):
        M, L = case["M"], case["L"]
        s["ids"] = _adapter_ids(g, M, L, case["runs"])
        s["order"] = torch.empty(M, dtype=torch.int32, device="cuda")
        s["offsets"] = torch.empty(L + 1, dtype=torch.int32, device="cuda")
        if case["op"] == "lora":
            K, N, R = case["K"], case["N"], case["R"]
            order, offsets = _group(s["ids"], L)
            s["order"].copy_(order)
            s["offsets"].copy_(offsets)
            s["x"] = _randn(g, M, K).to(torch.bfloat16)
            s["a"] = (_randn(g, L, R, K) * K ** -0.5).to(torch.bfloat16)
            s["b"] = (_randn(g, L, N, R) * 0.3).to(torch.bfloat16)
            s["scales"] = torch.rand(L, generator=g, device="cuda") + 0.5
            s["ranks"] = torch.tensor(_ranks(case), dtype=torch.int32, device="cuda")
            s["base"] = (_randn(g, M, N) * 2.0).to(torch.bfloat16)
            s["y"] = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    else:
        T, HQ, HK, D, rot = case["T"], case["HQ"], case["HK"], case["D"], case["rot"]
        qkv = (_randn(g, T, (HQ + 2 * HK) * D) * 2.0).to(torch.bfloat16)
        s["q"] = qkv[:, :HQ * D].view(T, HQ, D)
        s["k"] = qkv[:, HQ * D:(HQ + HK) * D].view(T, HK, D)
        s["gq"] = (1.0 + 0.2 * _randn(g, D)).to(torch.bfloat16)
        s["gk"] = (1.0 + 0.2 * _randn(g, D)).to(torch.bfloat16)
        freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        ang = torch.arange(case["P"], dtype=torch.float64, device="cuda")[:, None] * freq
        s["table"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        start = torch.randint(0, max(1, case["P"] - T + 1), (1,), generator=g, device="cuda")
        s["pos"] = (start + torch.arange(T, device="cuda")) % case["P"]
        s["qo"] = torch.empty(T, HQ, D, dtype=torch.bfloat16, device="cuda")
        s["ko"] = torch.empty(T, HK, D, dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_moe(s):
    import block_wise_fp8_gb300 as fb
    c = s["case"]
    if "ws" not in s:
        s["ws"] = fb.new_moe_workspace(c["M"], c["E"], c["H"], c["I"], c["topk"])
    fb.fp8bq_moe_layer(s["x"], s["logits"], s["w13"], s["s13"], s["w2"], s["s2"], s["y"], s["ws"],
                       c["topk"], score=fb.MOE_SOFTMAX if c["score"] == "softmax"
                       else fb.MOE_SIGMOID, renormalize=c["renorm"], routed_scale=c["scale"],
                       bias=s["bias"], ids_out=s["ids"], weights_out=s["weights"])
    return {"y": s["y"], "ids": s["ids"], "weights": s["weights"]}


def _own_lora(s):
    import block_wise_fp8_gb300 as fb
    c = s["case"]
    if "ws" not in s:
        s["ws"] = fb.new_workspace(fb.OP_LORA_ADD, c["M"], c["R"], c["K"])
    fb.fp8bq_lora_add(s["x"], s["a"], s["b"], s["scales"], s["order"], s["offsets"], s["base"],
                      s["y"], s["ws"], ranks=s["ranks"])
    return s["y"]


def _own_group(s):
    import block_wise_fp8_gb300 as fb
    fb.fp8bq_lora_group(s["ids"], s["order"], s["offsets"])
    return {"order": s["order"], "offsets": s["offsets"]}


def _own_rope(s):
    import block_wise_fp8_gb300 as fb
    fb.fp8bq_qk_norm_rope(s["q"], s["k"], s["gq"], s["gk"], s["table"], s["pos"], s["qo"], s["ko"],
                          eps=1e-6, interleaved=s["case"]["inter"])
    return {"q": s["qo"], "k": s["ko"]}


def _quant_rows(v):
    """Group-128 quantisation over the last axis, as the values the codes and
    scales stand for (binary32 divisions, nearest even, amax floored at 1e-10)."""
    K = v.shape[-1]
    pad = torch.nn.functional.pad(v, (0, -K % 128))
    grp = pad.reshape(*v.shape[:-1], -1, 128)
    s = grp.abs().amax(-1, keepdim=True).clamp(min=1e-10) / E4M3_MAX
    q = (grp / s).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).float()
    return (q * s).reshape(*v.shape[:-1], -1)[..., :K]


def _dequant(q, s):
    E, rows, cols = q.shape
    full = s.repeat_interleave(128, 1)[:, :rows].repeat_interleave(128, 2)[:, :, :cols]
    return q.float() * full


def _plain_moe(s):
    c = s["case"]
    topk, l = c["topk"], s["logits"]
    score = torch.softmax(l, -1) if c["score"] == "softmax" else torch.sigmoid(l)
    # the order of the chosen is that of the logits, which no rounding can turn;
    # with a bias it is that of sigmoid + bias, in 64 bits
    key = l if s["bias"] is None else torch.sigmoid(l.double()) + s["bias"].double()
    ids = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :topk]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    w = w * c["scale"]
    # every token through every expert, then the chosen experts' rows weighted
    I = c["I"]
    gu = torch.matmul(_quant_rows(s["x"].float()), _dequant(s["w13"], s["s13"]).transpose(1, 2))
    h = gu[..., :I] * torch.sigmoid(gu[..., :I]) * gu[..., I:]
    o = torch.matmul(_quant_rows(h), _dequant(s["w2"], s["s2"]).transpose(1, 2))
    rw = torch.zeros_like(l).scatter_(1, ids, w)
    y = (rw.t()[:, :, None] * o).sum(0)
    return {"y": y.to(torch.bfloat16), "ids": ids.to(torch.int32), "weights": w}


def _plain_lora(s):
    c = s["case"]
    M, L, R = c["M"], c["L"], c["R"]
    # every token through every adapter, masked to its own and to the rank
    t = s["x"].float() @ s["a"].float().reshape(L * R, -1).t()
    on = s["ids"][:, None, None] == torch.arange(L, device="cuda")[None, :, None]
    on = on & (torch.arange(R, device="cuda")[None, None, :] < s["ranks"][None, :, None])
    t = torch.where(on, t.view(M, L, R) * s["scales"][None, :, None], 0.0)
    d = t.view(M, L * R) @ s["b"].float().transpose(0, 1).reshape(c["N"], L * R).t()
    return (s["base"].float() + d).to(torch.bfloat16)


def _group(ids, L):
    key = torch.where((ids >= 0) & (ids < L), ids, L).long()
    order = torch.sort(key, stable=True).indices.to(torch.int32)
    counts = (key[:, None] == torch.arange(L, device="cuda")[None, :]).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    return order, offsets


def _plain_group(s):
    order, offsets = _group(s["ids"], s["case"]["L"])
    return {"order": order, "offsets": offsets}


def _plain_rope(s):
    c = s["case"]
    rot = c["rot"]
    cs = s["table"][s["pos"]][:, None, :]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]

    def one(v, gamma):
        v = v.float()
        v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + 1e-6) * gamma.float()
        r = v[..., :rot]
        if c["inter"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = r[..., :rot // 2], r[..., rot // 2:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([r, v[..., rot:]], -1).to(torch.bfloat16)

    return {"q": one(s["q"], s["gq"]), "k": one(s["k"], s["gk"])}


_OWN = {"moe": _own_moe, "lora": _own_lora, "group": _own_group, "rope": _own_rope}
_PLAIN = {"moe": _plain_moe, "lora": _plain_lora, "group": _plain_group, "rope": _plain_rope}


# ---------------------------------------------------------------- work

def work(case):
    if case["op"] == "moe":
        M, E, H, I, k = (case[n] for n in ("M", "E", "H", "I", "topk"))
        # experts that M independent choices of k reach, on average
        active = E * (1.0 - (1.0 - k / E) ** M)
        per = 3 * I * H + 4 * (3 * (-(-I // 128)) * (-(-H // 128)))
        return {"bytes": int(active * per + M * (4 * H + 4 * E + 8 * k)),
                "flops": 2 * M * k * 3 * I * H}
    if case["op"] == "lora":
        M, K, N, L = case["M"], case["K"], case["N"], case["L"]
        ranks = _ranks(case)
        runs = -(-M // case["runs"])
        share = min(1.0, runs / (L + 1.0))  # adapters that the runs reach
        mean = sum(ranks) / L
        return {"bytes": int(2 * M * K + 4 * M * N + 4 * M
                             + 2 * max(1.0, share * L) * mean * (K + N)),
                "flops": int(2 * M * mean * (K + N))}
    if case["op"] == "group":
        return {"bytes": 8 * case["M"] + 4 * case["L"] + 4, "flops": 0}
    n = case["T"] * (case["HQ"] + case["HK"]) * case["D"]
    return {"bytes": 4 * n + 4 * min(case["T"], case["P"]) * case["rot"] + 8 * case["T"],
            "flops": 7 * n}


# ---------------------------------------------------------------- 64 bits

def _e4m3_round(v):
    """Nearest E4M3 value of |v| <= 448, ties to even, in 64 bits."""
    e = torch.frexp(v)[1].double() - 1.0
    step = torch.exp2(e.clamp(min=-6.0) - 3.0)
    return torch.round(v / step) * step


def _exact_quant(v, binary32):
    """Group-128 quantisation of [rows, K]: codes' values times scales.  The
    activations' rule is stated in binary32 divisions; hidden rows are the
    formula's own values, so theirs are 64-bit ones."""
    n, K = v.shape
    out = torch.empty_like(v)
    for k0 in range(0, K, 128):
        blk = v[:, k0:k0 + 128]
        amax = blk.abs().max(1, keepdim=True).values.clamp(min=1e-10)
        if binary32:
            sc = (amax.float() / 448.0)
            ratio = (blk.float() / sc).double()
            sc = sc.double()
        else:
            sc = amax / 448.0
            ratio = blk / sc
        out[:, k0:k0 + 128] = _e4m3_round(ratio.clamp(-448.0, 448.0)) * sc
    return out


def _exact_weight(q, sc):
    rows, cols = q.shape
    i = torch.arange(rows, device="cuda") // 128
    j = torch.arange(cols, device="cuda") // 128
    return q.double() * sc.double()[i][:, j]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "moe":
        l = s["logits"].double()
        if case["score"] == "softmax":
            p = torch.exp(l - l.max(1, keepdim=True).values)
            p = p / p.sum(1, keepdim=True)
        else:
            p = 1.0 / (1.0 + torch.exp(-l))
        left = (l if s["bias"] is None else p + s["bias"].double()).clone()
        ids = []
        for _ in range(case["topk"]):
            best = left.max(1, keepdim=True).values
            first = (left == best).int().argmax(1)  # the lowest index of the largest
            ids.append(first)
            left.scatter_(1, first[:, None], -math.inf)
        ids = torch.stack(ids, 1)
        w = p.gather(1, ids)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        w = w * case["scale"]
        I = case["I"]
        xq = _exact_quant(s["x"].double(), True)
        y = torch.zeros(case["M"], case["H"], dtype=torch.float64, device="cuda")
        for e in range(case["E"]):
            tok, slot = (ids == e).nonzero(as_tuple=True)
            if tok.numel() == 0:
                continue
            gu = xq[tok] @ _exact_weight(s["w13"][e], s["s13"][e]).t()
            gate, up = gu[:, :I], gu[:, I:]
            h = _exact_quant(gate / (1.0 + torch.exp(-gate)) * up, False)
            o = h @ _exact_weight(s["w2"][e], s["s2"][e]).t()
            y.index_add_(0, tok, o * w[tok, slot][:, None])
        return {"y": y, "ids": ids.to(torch.int32), "weights": w}
    if case["op"] == "lora":
        y = s["base"].double()
        for a in range(case["L"]):
            tok = (s["ids"] == a).nonzero(as_tuple=True)[0]
            if tok.numel() == 0:
                continue
            r = int(s["ranks"][a])
            t = s["x"][tok].double() @ s["a"][a, :r].double().t()
            y[tok] += s["scales"][a].double() * (t @ s["b"][a, :, :r].double().t())
        return y
    if case["op"] == "group":
        return None
    rot, half = case["rot"], case["rot"] // 2
    cs = s["table"][s["pos"]].double()
    cos, sin = cs[:, None, :half], cs[:, None, half:]
    i = torch.arange(half, device="cuda")
    first, second = (2 * i, 2 * i + 1) if case["inter"] else (i, i + half)
    out = {}
    for n, v, gamma in (("q", s["q"], s["gq"]), ("k", s["k"], s["gk"])):
        v = v.double()
        v = v / torch.sqrt(v.pow(2).sum(-1, keepdim=True) / case["D"] + 1e-6) * gamma.double()
        z = v.clone()
        z[..., first] = v[..., first] * cos - v[..., second] * sin
        z[..., second] = v[..., second] * cos + v[..., first] * sin
        out[n] = z
    return out
