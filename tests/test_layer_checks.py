"""Refusals of the operators beside the linears, without a GPU: the binding's
checks (host tensors of the right shape fail only the device check) and the C
interface's host-side checks.  The fake addresses below are never launched with:
every call here is refused, or has no tokens, wherever it runs."""
import ctypes

import pytest
import torch

import block_wise_fp8_gb300 as fb

BF16, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
A = 0x100000  # a fake, aligned device address: the checks never follow it
OK, NULL, SHAPE, ALIGN, UNSUP, WORKSPACE = 0, 1, 2, 3, 4, 6


def z(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype)


def raises(match, fn, *a, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


# ---------------------------------------------------------------- binding

def rope(**kw):
    d = dict(q=z(3, 4, 64), k=z(3, 2, 64), q_gamma=z(64), k_gamma=z(64), table=z(16, 32, dtype=F32),
             positions=z(3, dtype=I64), q_out=z(3, 4, 64), k_out=z(3, 2, 64))
    d.update(kw)
    fb.fp8bq_qk_norm_rope(*d.values())


def test_rope_binding():
    raises("must be a CUDA tensor", rope)
    raises("must be a CUDA tensor", rope, k=None, k_out=None)
    raises("must be a CUDA tensor", rope, q=z(3, 400)[:, :256].view(3, 4, 64))
    raises("k_out without k|k_out must have shape", rope, k=None)
    raises("k_out is required", rope, k_out=None)
    raises("q must be a 3-D tensor", rope, q=z(3, 256))
    raises("q_out must have shape", rope, q_out=z(3, 4, 32))
    raises("k must have shape|must have shape", rope, k=z(2, 2, 64))
    raises("positions must be int32 or int64", rope, positions=z(3, dtype=F32))
    raises("positions must have shape", rope, positions=z(4, dtype=I64))
    raises("table must be float32", rope, table=z(16, 32))
    raises("unit stride", rope, q=z(3, 64, 4).transpose(1, 2))
    raises("q_gamma must have 64", rope, q_gamma=z(32))


def lora(**kw):
    d = dict(x=z(5, 64), a=z(3, 16, 64), b=z(3, 40, 16), scales=z(3, dtype=F32),
             order=z(5, dtype=I32), offsets=z(4, dtype=I32), base=z(5, 40), y=z(5, 40),
             ws=z(4096, dtype=torch.uint8), ranks=None)
    d.update(kw)
    fb.fp8bq_lora_add(*d.values())


def test_lora_binding():
    raises("must be a CUDA tensor", lora)
    raises("must be a CUDA tensor", lora, y=z(5, 60)[:, :40], x=z(5, 80)[:, :64])
    raises("a must be a 3-D", lora, a=z(16, 64))
    raises("a must have shape", lora, a=z(3, 16, 32))
    raises("b must have shape", lora, b=z(3, 16, 40))
    raises("order must be int32", lora, order=z(5, dtype=I64))
    raises("offsets must have shape", lora, offsets=z(3, dtype=I32))
    raises("scales must have shape", lora, scales=z(2, dtype=F32))
    raises("base must have shape", lora, base=z(5, 48))
    raises("ranks must have shape", lora, ranks=z(2, dtype=I32))
    raises("unit stride", lora, base=z(40, 5).t())


def test_group_binding():
    ids = z(5, dtype=I32)
    raises("must be a CUDA tensor", fb.fp8bq_lora_group, ids, ids.clone(), z(4, dtype=I32))
    raises("order must have shape", fb.fp8bq_lora_group, ids, z(4, dtype=I32), z(4, dtype=I32))
    raises("ids must be int32", fb.fp8bq_lora_group, z(5, dtype=I64), ids, z(4, dtype=I32))
    raises("L \\+ 1 elements", fb.fp8bq_lora_group, ids, ids, z(1, dtype=I32))


# ---------------------------------------------------------------- C interface

_lib = ctypes.CDLL(fb.library_path())
P, I, N, S, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float


def c_rope(q=A, HQ=4, k=A, HK=2, gq=A, gk=A, eps=1e-6, table=A, Pn=16, rot=32, pos=A, bits=64,
           qo=A, ko=A, T=3, D=64, ts=512, hs=64):
    return _lib.fp8bq_qk_norm_rope(P(q), I(ts), I(hs), I(HQ), P(k), I(ts), I(hs), I(HK), P(gq),
                                   P(gk), F(eps), P(table), I(Pn), I(rot), P(pos), N(bits), N(0),
                                   P(qo), I(ts), I(hs), P(ko), I(ts), I(hs), I(T), I(D), P(0))


def test_rope_abi():
    assert c_rope(T=0) == OK
    for kw in (dict(T=-1), dict(HQ=0, HK=0), dict(D=528), dict(D=0), dict(rot=80), dict(Pn=0),
               dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(HQ=-1)):
        assert c_rope(**kw) == SHAPE, kw
    for kw in (dict(D=72), dict(rot=24), dict(q=A + 8), dict(ko=A + 2), dict(gq=A + 4),
               dict(table=A + 4), dict(pos=A + 4), dict(ts=100), dict(hs=4)):
        assert c_rope(**kw) == ALIGN, kw
    for kw in (dict(q=0), dict(k=0), dict(qo=0), dict(ko=0), dict(pos=0), dict(table=0)):
        assert c_rope(**kw) == NULL, kw
    assert c_rope(bits=16) == UNSUP


def c_lora(x=A, ldx=64, a=A, b=A, sc=A, ranks=0, order=A, off=A, base=A, ldb=40, y=A, ldy=40, M=5,
           Nn=40, K=64, L=3, R=16, ws=A, wsb=1 << 20):
    return _lib.fp8bq_lora_add(P(x), I(ldx), P(a), P(b), P(sc), P(ranks), P(order), P(off), P(base),
                               I(ldb), P(y), I(ldy), I(M), I(Nn), I(K), I(L), I(R), P(ws), S(wsb),
                               P(0))


def test_lora_abi():
    assert c_lora(M=0, x=0, y=0, ws=0) == OK
    for kw in (dict(M=-1), dict(L=0), dict(L=513), dict(R=0), dict(R=136), dict(ldb=32),
               dict(ldy=32), dict(ldy=48), dict(ldx=48), dict(K=0), dict(Nn=0)):
        assert c_lora(**kw) == SHAPE, kw
    for kw in (dict(R=12), dict(K=56), dict(Nn=36), dict(ldb=44), dict(x=A + 2), dict(a=A + 8),
               dict(b=A + 8), dict(base=A + 4), dict(y=A + 4), dict(order=A + 2), dict(ws=A + 16),
               dict(ranks=A + 2)):
        assert c_lora(**kw) == ALIGN, kw
    for n in ("x", "a", "b", "sc", "order", "off", "base", "y"):
        assert c_lora(**{n: 0}) == NULL, n
    need = fb.fp8bq_workspace_bytes(fb.OP_LORA_ADD, 5, 16, 64)
    assert c_lora(wsb=need - 1) == WORKSPACE and c_lora(ws=0) == WORKSPACE


def test_group_abi():
    def c(ids=A, M=5, L=3, order=A, off=A):
        return _lib.fp8bq_lora_group(P(ids), I(M), I(L), P(order), P(off), P(0))
    assert c(M=-1) == SHAPE and c(L=0) == SHAPE and c(L=513) == SHAPE and c(M=2 ** 31 - 1) == SHAPE
    assert c(ids=0) == NULL and c(order=0) == NULL and c(off=0) == NULL
    assert c(ids=A + 2) == ALIGN and c(off=A + 1) == ALIGN


# ---------------------------------------------------------------- MoE layer

U8 = torch.uint8


def moe(fn=None, **kw):
    M, E, H, In, k = 5, 3, 272, 128, 2
    d = dict(x=z(M, H), logits=z(M, E, dtype=F32), w13=z(E, 2 * In, H, dtype=U8),
             s13=z(E, 2, 3, dtype=F32), w2=z(E, H, In, dtype=U8), s2=z(E, 3, 1, dtype=F32),
             y=z(M, H), ws=z(4096, dtype=U8), topk=k)
    d.update(kw)
    fb.fp8bq_moe_layer(**d)


def test_moe_binding():
    raises("must be a CUDA tensor", moe)
    raises("must be a CUDA tensor", moe, x=z(5, 300)[:, :272], ids_out=z(5, 2, dtype=I32))
    raises("logits must have shape", moe, logits=z(5, 4, dtype=F32))
    raises("logits must be float32", moe, logits=z(5, 3))
    raises("w13 must have shape", moe, w13=z(3, 255, 272, dtype=U8))
    raises("3-D", moe, w13=z(256, 272, dtype=U8))
    raises("s13 must have shape", moe, s13=z(3, 3, 2, dtype=F32))
    raises("w2 must have shape", moe, w2=z(3, 128, 272, dtype=U8))
    raises("s2 must have shape", moe, s2=z(3, 1, 3, dtype=F32))
    raises("y must have shape", moe, y=z(5, 256))
    raises("bias must have shape", moe, bias=z(4, dtype=F32))
    raises("ids_out must have shape", moe, ids_out=z(5, 3, dtype=I32))
    raises("weights_out must be float32", moe, weights_out=z(5, 2))
    raises("ws is required", moe, ws=None)


def test_moe_experts_binding():
    a = (z(3, 256, 272, dtype=U8), z(3, 2, 3, dtype=F32), z(3, 272, 128, dtype=U8),
         z(3, 3, 1, dtype=F32), z(5, 272), z(4096, dtype=U8))
    ok = (z(5, 272), z(5, 2, dtype=I32), z(5, 2, dtype=F32))
    raises("must be a CUDA tensor", fb.fp8bq_moe_experts, *ok, *a)
    raises("weights must have shape", fb.fp8bq_moe_experts, ok[0], ok[1], z(5, 3, dtype=F32), *a)
    raises("ids must have shape", fb.fp8bq_moe_experts, ok[0], z(4, 2, dtype=I32), ok[2], *a)


_lib.fp8bq_moe_workspace_bytes.restype = S


def c_moe(x=A, ldx=256, lg=A, bias=0, score=0, topk=2, w13=A, s13=A, w2=A, s2=A, y=A, io=0, wo=0,
          M=5, E=4, H=256, In=128, ws=A, wsb=1 << 30):
    return _lib.fp8bq_moe_layer(P(x), I(ldx), P(lg), P(bias), N(score), N(1), F(1.0), I(topk),
                                P(w13), P(s13), P(w2), P(s2), P(y), P(io), P(wo), I(M), I(E), I(H),
                                I(In), P(ws), S(wsb), P(0))


def test_moe_abi():
    assert c_moe(M=0, x=0, lg=0) == OK
    assert c_moe(M=65) == UNSUP and c_moe(score=2) == UNSUP and c_moe(bias=A) == UNSUP
    assert c_moe(score=1, bias=A, ws=0) == WORKSPACE  # the last check: all others passed
    for kw in (dict(M=-1), dict(E=0), dict(E=513), dict(topk=0), dict(topk=5), dict(topk=17, E=64),
               dict(H=0), dict(In=0), dict(ldx=128), dict(H=65552), dict(In=65664)):
        assert c_moe(**kw) == SHAPE, kw
    for kw in (dict(H=248), dict(In=64), dict(x=A + 8), dict(w13=A + 8), dict(w2=A + 8),
               dict(y=A + 8), dict(s13=A + 2), dict(s2=A + 2), dict(lg=A + 1), dict(io=A + 1),
               dict(ws=A + 128), dict(ldx=260)):
        assert c_moe(**kw) == ALIGN, kw
    for n in ("x", "lg", "w13", "s13", "w2", "s2", "y"):
        assert c_moe(**{n: 0}) == NULL, n
    need = fb.fp8bq_moe_workspace_bytes(5, 4, 256, 128, 2)
    assert c_moe(wsb=need - 1) == WORKSPACE and c_moe(ws=0) == WORKSPACE
    assert fb.fp8bq_moe_workspace_bytes(65, 4, 256, 128, 2) == 256


def test_moe_experts_abi():
    def c(ids=A, w=A, M=5, topk=2):
        return _lib.fp8bq_moe_experts(P(A), I(256), P(ids), P(w), I(topk), P(A), P(A), P(A), P(A),
                                      P(A), I(M), I(4), I(256), I(128), P(A), S(1 << 30), P(0))
    assert c(M=0, ids=0) == OK
    assert c(ids=0) == NULL and c(w=0) == NULL and c(ids=A + 2) == ALIGN and c(topk=17) == SHAPE


def test_rope_outputs_whose_heads_overlap():
    """4 query and 2 key heads of 64 values, 3 tokens; what overlaps is refused
    whatever the order of the strides (inputs may: q's and k's strides go along)."""
    for kw in (dict(ts=64), dict(ts=0), dict(hs=0), dict(hs=56), dict(ts=248), dict(ts=-248),
               dict(ts=-64, hs=64), dict(ts=64, hs=184), dict(ts=96, hs=128), dict(T=1, hs=48),
               dict(HQ=1, HK=1, ts=56), dict(HK=0, k=0, ko=0, hs=0)):
        assert c_rope(**kw) == SHAPE, kw
