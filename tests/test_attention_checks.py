"""Refusals of the attention operators and of their cache, without a GPU: the binding's
checks and the C interface's host-side checks.  The fake addresses below are never
launched with: every call here is refused, or has nothing to do, wherever it runs."""
import ctypes

import pytest
import torch

import block_wise_fp8_gb300 as fb

BF16, F32, I32, I64, U8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8
A = 0x100000  # a fake, aligned device address: the checks never follow it
OK, NULL, SHAPE, ALIGN, UNSUP, WORKSPACE = 0, 1, 2, 3, 4, 6
NAN, INF = float("nan"), float("inf")


def z(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype)


def raises(match, fn, *a, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


# ---------------------------------------------------------------- binding

def prompt(**kw):
    d = dict(q=z(5, 4, 64), k=z(5, 2, 64), v=z(5, 2, 64), offsets=z(3, dtype=I32), y=z(5, 4, 64),
             ws=z(256, dtype=U8))
    d.update(kw)
    fb.fp8bq_prompt_attention(**d)


def test_prompt_binding():
    raises("must be a CUDA tensor", prompt)
    raises("must be a CUDA tensor", prompt, q=z(5, 512)[:, :256].view(5, 4, 64))
    raises("q must be a 3-D", prompt, q=z(5, 256))
    raises("k must be a 3-D", prompt, k=None)
    raises("v must have shape", prompt, v=z(5, 3, 64))
    raises("k must have shape", prompt, k=z(4, 2, 64))
    raises("y must have shape", prompt, y=z(5, 4, 32))
    raises("y must be bfloat16", prompt, y=z(5, 4, 64, dtype=F32))
    raises("offsets must be", prompt, offsets=z(3, dtype=I64))
    raises("offsets must be", prompt, offsets=None)
    raises("unit stride", prompt, v=z(5, 64, 2).transpose(1, 2))
    raises("ws must be|ws is required", prompt, ws=None)


def rows(fn, **kw):
    d = dict(k=z(3, 2, 64), v=z(3, 2, 64), slots=z(3, dtype=I32), cache=z(4, 2, 16 * 72, dtype=U8))
    d.update(kw)
    fn(**d)


@pytest.mark.parametrize("fn", [fb.fp8bq_kv4_append, fb.fp8bq_kv4_read])
def test_rows_binding(fn):
    raises("must be a CUDA tensor", rows, fn)
    raises("must be a CUDA tensor", rows, fn, slots=z(3, dtype=I64))
    raises("k must be a 3-D", rows, fn, k=z(3, 128))
    raises("v must have shape", rows, fn, v=z(3, 2, 32))
    raises("slots must be int32 or int64", rows, fn, slots=z(3, dtype=F32))
    raises("slots must have shape", rows, fn, slots=z(4, dtype=I32))
    raises("no page of", rows, fn, cache=z(4, 2, 16 * 72 + 1, dtype=U8))
    raises("no page of", rows, fn, cache=z(4, 2, 8 * 72, dtype=U8))
    raises("cache must be a 3-D", rows, fn, cache=z(4, 16 * 72, dtype=U8))
    raises("cache must be uint8", rows, fn, cache=z(4, 2, 16 * 72, dtype=torch.int8))
    raises("the cache has 3 heads", rows, fn, cache=z(4, 3, 16 * 72, dtype=U8))
    raises("must be contiguous", rows, fn, cache=z(4, 4, 16 * 72, dtype=U8)[:, ::2])


def test_append_weights_binding():
    raises("weights must have shape", rows, fb.fp8bq_kv4_append, weights=z(4, 2, 32, dtype=F32))
    raises("weights must be float32", rows, fb.fp8bq_kv4_append, weights=z(4, 2, 16))


def attend(**kw):
    d = dict(q=z(6, 4, 64), cache=z(8, 2, 16 * 72, dtype=U8), table=z(3, 2, dtype=I32),
             lens=z(3, dtype=I32), y=z(6, 4, 64), ws=z(4096, dtype=U8),
             weights=z(8, 2, 16, dtype=F32))
    d.update(kw)
    fb.fp8bq_kv4_attention(**d)


def test_attention_binding():
    raises("must be a CUDA tensor", attend)
    raises("must be a CUDA tensor", attend, weights=None)
    raises("6 rows for 4 sequences", attend, table=z(4, 2, dtype=I32))
    raises("6 rows for 0 sequences", attend, table=z(0, 2, dtype=I32))
    raises("table must be a 2-D", attend, table=z(3, dtype=I32))
    raises("table must be int32", attend, table=z(3, 2, dtype=I64))
    raises("lens must have shape", attend, lens=z(2, dtype=I32))
    raises("y must have shape", attend, y=z(6, 2, 64))
    raises("weights must have shape", attend, weights=z(8, 2, 32, dtype=F32))
    raises("cache must be a 3-D", attend, cache=None)
    raises("no page of", attend, q=z(6, 4, 128))


def evict(**kw):
    d = dict(cache=z(8, 2, 16 * 72, dtype=U8), table=z(3, 2, dtype=I32), lens=z(3, dtype=I32),
             weights=z(8, 2, 16, dtype=F32), new_table=z(3, 1, dtype=I32), new_lens=z(3, dtype=I32),
             kept=z(3, 2, 9, dtype=I32), recent=3, D=64)
    d.update(kw)
    fb.fp8bq_kv4_evict(**d)


def test_evict_binding():
    raises("must be a CUDA tensor", evict)
    raises("weights is required", evict, weights=None)
    raises("new_table must have shape", evict, new_table=z(2, 1, dtype=I32))
    raises("new_lens must be int32", evict, new_lens=z(3, dtype=I64))
    raises("kept must have shape", evict, kept=z(3, 1, 9, dtype=I32))
    raises("kept must be a 3-D", evict, kept=z(3, 18, dtype=I32))
    raises("no page of", evict, D=0)


def test_new_cache():
    assert fb.new_kv4_cache(3, 2, 32, 128, device="cpu").shape == (3, 2, 32 * 144)
    raises("page must be", fb.new_kv4_cache, 3, 2, 8, 128, device="cpu")
    raises("page must be", fb.new_kv4_cache, 3, 2, 16, 96, device="cpu")


# ---------------------------------------------------------------- C interface

def c_prompt(**kw):
    d = dict(q=A, q_ts=512, q_hs=64, k=A, k_ts=512, k_hs=64, v=A, v_ts=512, v_hs=64, offsets=A, S=2,
             scale=0.1, y=A, y_ts=256, y_hs=64, T=10, HQ=4, HK=2, D=64, ws=A, ws_bytes=256, stream=0)
    d.update(kw)
    return fb._lib.fp8bq_prompt_attention(*d.values())


def test_prompt_c():
    for bad in (dict(T=-1), dict(T=2 ** 19 + 1), dict(S=-1), dict(S=1025), dict(HK=0), dict(HQ=5),
                dict(HQ=0), dict(HQ=2048), dict(scale=0.0), dict(scale=-1.0), dict(scale=NAN),
                dict(scale=INF), dict(q_ts=0), dict(k_hs=-64), dict(y_ts=64), dict(y_hs=0)):
        assert c_prompt(**bad) == SHAPE, bad
    for bad in (dict(D=8), dict(D=144), dict(HQ=258, HK=2)):
        assert c_prompt(**bad) == UNSUP, bad
    for bad in (dict(D=72), dict(q=A + 8), dict(k=A + 2), dict(v=A + 8), dict(y=A + 8), dict(q_ts=516),
                dict(v_hs=60), dict(offsets=A + 2), dict(ws=A + 16)):
        assert c_prompt(**bad) == ALIGN, bad
    for bad in (dict(q=0), dict(k=0), dict(v=0), dict(offsets=0), dict(y=0)):
        assert c_prompt(**bad) == NULL, bad
    assert c_prompt(ws=0) == WORKSPACE and c_prompt(ws_bytes=255) == WORKSPACE
    assert c_prompt(T=0, q=0, k=0, v=0, y=0) == OK
    assert c_prompt(S=0) == OK
    assert fb.fp8bq_workspace_bytes(fb.OP_PROMPT_ATTENTION, 10, 4, 64) == 256


def c_append(**kw):
    d = dict(k=A, k_ts=512, k_hs=64, v=A, v_ts=512, v_hs=64, slots=A, slot_bits=32, cache=A, pages=4,
             page=16, weights=0, k_scale=1.0, v_scale=1.0, T=3, HK=2, D=64, stream=0)
    d.update(kw)
    return fb._lib.fp8bq_kv4_append(*d.values())


def c_read(**kw):
    d = dict(cache=A, pages=4, page=16, slots=A, slot_bits=32, k_scale=1.0, v_scale=1.0, k=A,
             k_ts=512, k_hs=64, v=A, v_ts=512, v_hs=64, T=3, HK=2, D=64, stream=0)
    d.update(kw)
    return fb._lib.fp8bq_kv4_read(*d.values())


@pytest.mark.parametrize("call", [c_append, c_read])
def test_rows_c(call):
    for bad in (dict(T=-1), dict(pages=0), dict(pages=2 ** 31), dict(HK=0), dict(HK=2000),
                dict(k_scale=0.0), dict(v_scale=NAN), dict(k_scale=INF), dict(v_scale=-1.0),
                dict(T=2 ** 31)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(page=8), dict(page=256), dict(page=48), dict(D=32), dict(D=96),
                dict(slot_bits=16)):
        assert call(**bad) == UNSUP, bad
    for bad in (dict(k=A + 8), dict(v=A + 2), dict(cache=A + 8), dict(slots=A + 2), dict(k_ts=516),
                dict(slot_bits=64, slots=A + 4)):
        assert call(**bad) == ALIGN, bad
    for bad in (dict(k=0), dict(v=0), dict(slots=0), dict(cache=0)):
        assert call(**bad) == NULL, bad
    assert call(T=0, k=0, v=0, slots=0) == OK


def test_read_rows_overlap_c():
    assert c_read(k_ts=64) == SHAPE and c_read(v_hs=0) == SHAPE
    assert c_append(weights=A + 2) == ALIGN


def c_attend(**kw):
    d = dict(q=A, q_ts=256, q_hs=64, cache=A, pages=8, page=16, table=A, width=2, lens=A, scale=0.1,
             k_scale=1.0, v_scale=1.0, weights=0, y=A, y_ts=256, y_hs=64, B=3, Tq=2, HQ=4, HK=2, D=64,
             ws=A, ws_bytes=1 << 30, stream=0)
    d.update(kw)
    return fb._lib.fp8bq_kv4_attention(*d.values())


def test_attention_c():
    for bad in (dict(B=-1), dict(B=1025), dict(Tq=0), dict(HQ=5), dict(HQ=0), dict(HK=0), dict(width=-1),
                dict(width=2 ** 28), dict(scale=0.0), dict(scale=NAN), dict(k_scale=0.0),
                dict(v_scale=INF), dict(pages=0), dict(y_ts=128), dict(scale=3e38, k_scale=3e38),
                dict(B=1024, HK=64, HQ=64)):
        assert c_attend(**bad) == SHAPE, bad
    for bad in (dict(page=24), dict(D=80), dict(Tq=65), dict(HQ=260, HK=2), dict(Tq=200)):
        assert c_attend(**bad) == UNSUP, bad
    for bad in (dict(q=A + 8), dict(cache=A + 8), dict(y=A + 8), dict(table=A + 2), dict(lens=A + 1),
                dict(weights=A + 2), dict(q_hs=60), dict(ws=A + 64)):
        assert c_attend(**bad) == ALIGN, bad
    for bad in (dict(q=0), dict(cache=0), dict(table=0), dict(lens=0), dict(y=0)):
        assert c_attend(**bad) == NULL, bad
    need = fb.fp8bq_kv4_workspace_bytes(3, 2, 4, 2, 64, 32)
    more = fb.fp8bq_kv4_workspace_bytes(3, 2, 4, 2, 64, 32, True)
    assert more > need and need % 256 == 0 and more % 256 == 0
    assert c_attend(ws_bytes=need - 1) == WORKSPACE and c_attend(ws=0) == WORKSPACE
    assert c_attend(ws_bytes=more - 1, weights=A) == WORKSPACE
    assert c_attend(B=0, q=0) == OK
    assert fb.fp8bq_kv4_workspace_bytes(3, 2, 5, 2, 64, 32) == 256


def c_evict(**kw):
    d = dict(cache=A, pages=8, page=16, table=A, width=4, lens=A, weights=A, new_table=A, new_width=2,
             new_lens=A + 64, kept=A, budget=20, recent=5, B=3, HK=2, D=64, stream=0)
    d.update(kw)
    return fb._lib.fp8bq_kv4_evict(*[ctypes.c_void_p(v) for v in d.values()])


def test_evict_c():
    for bad in (dict(B=-1), dict(B=1025), dict(width=-1), dict(budget=0), dict(recent=-1), dict(recent=21),
                dict(new_width=1), dict(new_lens=A), dict(budget=33), dict(HK=0)):
        assert c_evict(**bad) == SHAPE, bad
    for bad in (dict(page=12), dict(D=192)):
        assert c_evict(**bad) == UNSUP, bad
    for bad in (dict(cache=A + 8), dict(table=A + 2), dict(lens=A + 2), dict(weights=A + 2),
                dict(new_table=A + 2), dict(new_lens=A + 2), dict(kept=A + 2)):
        assert c_evict(**bad) == ALIGN, bad
    for bad in (dict(cache=0), dict(table=0), dict(lens=0), dict(weights=0), dict(new_table=0),
                dict(new_lens=0), dict(kept=0)):
        assert c_evict(**bad) == NULL, bad
    assert c_evict(B=0, lens=0) == OK
