"""One decode step of a block-FP8 decoder layer, out of the library's calls:

    residual add + RMSNorm + quantisation   fp8bq_add_rmsnorm_quant_act
    QKV projection, adapters beside it      fp8bq_gemm, fp8bq_lora_add
    head norms and rotary embedding         fp8bq_qk_norm_rope
    attention                               plain torch over BF16 rows, or with
                                            cache4=True fp8bq_kv4_append and
                                            fp8bq_kv4_attention over a paged cache in
                                            4 bits; whole prompts (offsets given):
                                            fp8bq_prompt_attention
    output projection, adapters             fp8bq_linear, fp8bq_lora_add
    residual add + RMSNorm                  fp8bq_add_rmsnorm_quant_act
    mixture of experts                      fp8bq_moe_layer

Every request has its own adapter (or none); the tokens are grouped by adapter
once a step.  With a 4-bit cache the softmax weight that each cached token gets is
added up, and `evict` keeps the heaviest and the last ones.
`python examples/decoder_layer.py` times the step on a GPU and prints how far it is
from the same layer in 64 bits with unquantised activations.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_wise_fp8_gb300 as fb  # noqa: E402

BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
SIZES = dict(H=2048, heads=16, kv_heads=2, D=128, E=32, I=512, topk=4, adapters=8, rank=16)


class Layer:
    """Weights, quantised once, and the buffers of a step of `M` tokens."""

    def __init__(self, M: int, seed: int = 0, H=2048, heads=16, kv_heads=2, D=128, E=32, I=512,
                 topk=4, adapters=8, rank=16, context=256, cache4=False, page=32):
        g = torch.Generator("cuda").manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.M, self.H, self.heads, self.kv, self.D = M, H, heads, kv_heads, D
        self.topk = topk
        nq, nqkv = heads * D, (heads + 2 * kv_heads) * D
        self.g1, self.g2 = [(1 + 0.1 * rn(H)).to(BF16) for _ in range(2)]
        self.gq, self.gk = [(1 + 0.1 * rn(D)).to(BF16) for _ in range(2)]
        self.qkv_w, self.qkv_s = self._quantise(rn(nqkv, H) * H ** -0.5)
        self.o_w, self.o_s = self._quantise(rn(H, nq) * nq ** -0.5)
        w13 = [self._quantise(rn(2 * I, H) * H ** -0.5) for _ in range(E)]
        w2 = [self._quantise(rn(H, I) * I ** -0.5) for _ in range(E)]
        self.w13, self.s13 = [torch.stack(t) for t in zip(*w13)]
        self.w2, self.s2 = [torch.stack(t) for t in zip(*w2)]
        self.router = rn(E, H) * H ** -0.5
        adapter = lambda K, N: ((rn(adapters, rank, K) * K ** -0.5).to(BF16),  # noqa: E731
                                (rn(adapters, N, rank) * 0.1).to(BF16))
        self.qkv_lora, self.o_lora = adapter(H, nqkv), adapter(nq, H)
        self.scales = torch.full((adapters,), 0.5, device="cuda")
        freq = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
        ang = torch.arange(4096, dtype=torch.float64, device="cuda")[:, None] * freq
        self.table = torch.cat([ang.cos(), ang.sin()], 1).float()
        # what the requests have cached: context rows of rotated keys and values
        self.k_cache = rn(M, context, kv_heads, D).to(BF16)
        self.v_cache = rn(M, context, kv_heads, D).to(BF16)
        e = lambda *s, dtype=BF16: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        self.resid1, self.resid2, self.n1, self.n2 = e(M, H), e(M, H), e(M, H), e(M, H)
        self.q8, self.q8s = e(M, H, dtype=U8), e(M, -(-H // 128), dtype=F32)
        self.qkv, self.q, self.k = e(M, nqkv), e(M, heads, D), e(M, kv_heads, D)
        self.attn, self.o, self.y = e(M, nq), e(M, H), e(M, H)
        self.order, self.offsets = e(M, dtype=I32), e(adapters + 1, dtype=I32)
        self.cache4 = None
        if cache4:
            self._new_cache(context, page)
        self.ws_prompt = fb.new_workspace(fb.OP_PROMPT_ATTENTION, M, heads, D)
        self.ws_qkv = fb.new_workspace(fb.OP_GEMM, M, nqkv, H)
        self.ws_o = fb.new_workspace(fb.OP_LINEAR, M, H, nq)
        lora = max(fb.fp8bq_workspace_bytes(fb.OP_LORA_ADD, M, rank, k) for k in (H, nq))
        self.ws_lora = torch.zeros(lora, dtype=U8, device="cuda")
        self.ws_moe = fb.new_moe_workspace(M, E, H, I, topk)

    @staticmethod
    def _quantise(w):
        w = w.to(BF16)
        q = torch.empty(w.shape, dtype=torch.float8_e4m3fn, device="cuda")
        s = torch.empty(-(-w.shape[0] // 128), -(-w.shape[1] // 128), device="cuda")
        fb.fp8bq_quant_weight_block(w, q, s)
        return q, s

    # ------------------------------------------------------------ the 4-bit cache

    def _new_cache(self, context, page, spare=64):
        """A cache with room for `context` rows of every request and `spare` more, its
        pages in no order, holding what k_cache and v_cache hold."""
        M, self.page = self.M, page
        width = -(-(context + spare) // page)
        self.cache4 = fb.new_kv4_cache(2 * M * width, self.kv, page, self.D)
        self.weights = torch.zeros(2 * M * width, self.kv, page, device="cuda")
        order = torch.randperm(2 * M * width, device="cuda").to(I32)
        self.pages, self.free = order[:M * width].view(M, width), order[M * width:].view(M, width)
        self.lens = torch.full((M,), context, dtype=I32, device="cuda")
        self.ws_kv4 = fb.new_kv4_workspace(M, 1, self.heads, self.kv, self.D, width * page, True)
        at = torch.arange(context, device="cuda").repeat(M, 1)
        self.write_rows(self.k_cache.flatten(0, 1), self.v_cache.flatten(0, 1),
                        self.slots(torch.arange(M, device="cuda")[:, None], at).flatten())

    def slots(self, request, at):
        """Slots of the requests' tokens `at`, by the block table; -1, which a write leaves
        out, behind its end."""
        width = self.pages.shape[1]
        pages = self.pages.long()[request, (at // self.page).clamp(max=width - 1)]
        return torch.where(at < width * self.page, pages * self.page + at % self.page, -1)

    def write_rows(self, k, v, slots):
        fb.fp8bq_kv4_append(k, v, slots, self.cache4, weights=self.weights)

    def read_rows(self, slots):
        k, v = [torch.empty(slots.numel(), self.kv, self.D, dtype=BF16, device="cuda")
                for _ in range(2)]
        fb.fp8bq_kv4_read(self.cache4, slots, k, v)
        return k, v

    def _attend4(self, q, k, v):
        """One new token a request: into the cache, then attention over all of it."""
        self.write_rows(k, v, self.slots(torch.arange(self.M, device="cuda"), self.lens.long()))
        fb.fp8bq_kv4_attention(q, self.cache4, self.pages, self.lens + 1,
                               self.attn.view(self.M, self.heads, self.D), self.ws_kv4,
                               weights=self.weights)

    def evict(self, budget, recent):
        """Keeps `budget` of each request's tokens a head, in the spare pages."""
        lens, kept = torch.empty_like(self.lens), torch.empty(self.M, self.kv, budget, dtype=I32,
                                                              device="cuda")
        fb.fp8bq_kv4_evict(self.cache4, self.pages, self.lens, self.weights, self.free, lens, kept,
                           recent, self.D)
        self.pages, self.free, self.lens = self.free, self.pages, lens
        return kept

    # ------------------------------------------------------------ a step

    def _attend(self, q, k, v, kc, vc):
        """Plain attention of one new token a request over its context."""
        k = torch.cat([kc, k[:, None]], 1).repeat_interleave(self.heads // self.kv, 2)
        v = torch.cat([vc, v[:, None]], 1).repeat_interleave(self.heads // self.kv, 2)
        p = torch.softmax(torch.einsum("mhd,mthd->mht", q, k) * self.D ** -0.5, -1)
        return torch.einsum("mht,mthd->mhd", p, v).reshape(self.M, -1)

    def _attend_prompts(self, q, k, v, bounds):
        """Plain causal attention of whole prompts, rows bounds[i] .. bounds[i+1]-1 each."""
        k, v = [t.repeat_interleave(self.heads // self.kv, 1) for t in (k, v)]
        y = torch.zeros_like(q)
        for a, b in zip(bounds, bounds[1:]):
            s = torch.einsum("ihd,jhd->hij", q[a:b], k[a:b]) * self.D ** -0.5
            s = s.masked_fill(torch.ones_like(s).triu(1).bool(), float("-inf"))
            y[a:b] = torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), v[a:b])
        return y.reshape(self.M, -1)

    def step(self, x, residual, positions, adapter_ids, offsets=None):
        """x, residual [M, H] BF16 -> the layer's output and new residual.  The rows are
        one new token of each request, or with `offsets` (int32 [S + 1]) whole prompts."""
        fb.fp8bq_lora_group(adapter_ids, self.order, self.offsets)
        fb.fp8bq_add_rmsnorm_quant_act(x, self.g1, 1e-6, residual=residual,
                                       residual_out=self.resid1, y=self.n1, q=self.q8, s=self.q8s)
        fb.fp8bq_gemm(self.q8, self.q8s, self.qkv_w, self.qkv_s, self.qkv, self.ws_qkv)
        self._adapters(self.n1, self.qkv_lora, self.qkv)
        nq, nk = self.heads * self.D, self.kv * self.D
        q = self.qkv[:, :nq].view(self.M, self.heads, self.D)
        k = self.qkv[:, nq:nq + nk].view(self.M, self.kv, self.D)
        v = self.qkv[:, nq + nk:].view(self.M, self.kv, self.D)
        fb.fp8bq_qk_norm_rope(q, k, self.gq, self.gk, self.table, positions, self.q, self.k)
        if offsets is not None:
            fb.fp8bq_prompt_attention(self.q, self.k, v, offsets,
                                      self.attn.view(self.M, self.heads, self.D), self.ws_prompt)
        elif self.cache4 is not None:
            self._attend4(self.q, self.k, v)
        else:
            self.attn.copy_(self._attend(self.q.float(), self.k.float(), v.float(),
                                         self.k_cache.float(), self.v_cache.float()))
        fb.fp8bq_linear(self.attn, self.o_w, self.o_s, self.o, self.ws_o)
        self._adapters(self.attn, self.o_lora, self.o)
        fb.fp8bq_add_rmsnorm_quant_act(self.o, self.g2, 1e-6, residual=self.resid1,
                                       residual_out=self.resid2, y=self.n2)
        logits = self.n2.float() @ self.router.t()
        fb.fp8bq_moe_layer(self.n2, logits, self.w13, self.s13, self.w2, self.s2, self.y,
                           self.ws_moe, self.topk)
        return self.y, self.resid2

    def _adapters(self, x, lora, y):
        fb.fp8bq_lora_add(x, *lora, self.scales, self.order, self.offsets, y, y, self.ws_lora)

    # ------------------------------------------------------------ 64 bits

    def reference(self, x, residual, positions, adapter_ids, offsets=None):
        """The same layer in 64 bits from the quantised weights, its activations
        not quantised.  The experts are those that the step's own norm output
        chooses, so that a close choice cannot differ.  With a 4-bit cache, keys and
        values are those that the step has left in it (of equal lengths)."""
        d = torch.float64
        deq = lambda q, s: q.to(d) * s.to(d).repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(  # noqa: E731
            128, 1)[:, :q.shape[1]]
        norm = lambda v, gain: v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6) * gain.to(d)  # noqa: E731

        def adapters(v, lora):
            a, b = lora
            on = (adapter_ids >= 0)[:, None].to(d)
            i = adapter_ids.clamp(min=0).long()
            t = torch.einsum("mk,mrk->mr", v, a.to(d)[i])
            return on * self.scales.to(d)[i][:, None] * torch.einsum("mr,mnr->mn", t, b.to(d)[i])

        r1 = x.to(d) + residual.to(d)
        n1 = norm(r1, self.g1)
        qkv = n1 @ deq(self.qkv_w, self.qkv_s).t() + adapters(n1, self.qkv_lora)
        nq, nk = self.heads * self.D, self.kv * self.D
        cs = self.table[positions].to(d)[:, None]
        c, s = cs[..., :self.D // 2], cs[..., self.D // 2:]

        def rotate(v, gain):
            v = norm(v, gain)
            a, b = v[..., :self.D // 2], v[..., self.D // 2:]
            return torch.cat([a * c - b * s, b * c + a * s], -1)

        q = rotate(qkv[:, :nq].view(self.M, self.heads, self.D), self.gq)
        k = rotate(qkv[:, nq:nq + nk].view(self.M, self.kv, self.D), self.gk)
        v = qkv[:, nq + nk:].view(self.M, self.kv, self.D)
        if offsets is not None:
            at = self._attend_prompts(q, k, v, offsets.tolist())
        elif self.cache4 is not None:
            n = int(self.lens[0])
            rows = self.read_rows(self.slots(torch.arange(self.M, device="cuda")[:, None],
                                             torch.arange(n + 1, device="cuda")[None]).flatten())
            kc, vc = [r.to(d).view(self.M, n + 1, self.kv, self.D) for r in rows]
            at = self._attend(q, kc[:, n], vc[:, n], kc[:, :n], vc[:, :n])
        else:
            at = self._attend(q, k, v, self.k_cache.to(d), self.v_cache.to(d))
        r2 = r1 + at @ deq(self.o_w, self.o_s).t() + adapters(at, self.o_lora)
        n2 = norm(r2, self.g2)
        logits = self.n2.float() @ self.router.t()
        top = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :self.topk]
        w = torch.softmax((n2 @ self.router.to(d).t()).gather(1, top), -1)
        y = torch.zeros_like(n2)
        for m in range(self.M):
            for j in range(self.topk):
                e = int(top[m, j])
                gu = deq(self.w13[e], self.s13[e]) @ n2[m]
                gate, up = gu.chunk(2)
                y[m] += w[m, j] * (deq(self.w2[e], self.s2[e]) @ (torch.nn.functional.silu(gate) * up))
        return y, r2


def inputs(layer: Layer, seed: int = 1, adapters: int = 8):
    g = torch.Generator("cuda").manual_seed(seed)
    M, H = layer.M, layer.H
    return (torch.randn(M, H, generator=g, device="cuda").to(BF16),
            torch.randn(M, H, generator=g, device="cuda").to(BF16),
            torch.randint(0, 4096, (M,), generator=g, device="cuda"),
            torch.randint(-1, adapters, (M,), generator=g, device="cuda", dtype=I32))


def main():
    for M, cache4 in ((1, False), (16, False), (64, False), (1, True), (16, True), (64, True)):
        layer = Layer(M, cache4=cache4, **SIZES)
        args = inputs(layer)
        y, r = layer.step(*args)
        ry, rr = layer.reference(*args)
        assert fb.fp8bq_poll_status(layer.ws_moe) == 0
        err = [float((a.double() - b).norm() / b.norm()) for a, b in ((y, ry), (r, rr))]
        start, end = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        start.record()
        for _ in range(50):
            layer.step(*args)
        end.record()
        torch.cuda.synchronize()
        print(f"{M:3d} tokens{', 4-bit cache' if cache4 else ''}: "
              f"{start.elapsed_time(end) * 20:.0f} us a step; relative error of the "
              f"output {err[0]:.3f}, of the residual {err[1]:.4f}")


if __name__ == "__main__":
    main()
