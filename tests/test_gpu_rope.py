"""Norm of query and key heads with the rotary embedding against the formulas
in 64 bits.  The kernel works in binary32 and rounds once to BF16, so a value
is off by at most half a BF16 step (2^-8 of it) plus the binary32 arithmetic:
the sum of D squares, a root, four products and a sum, (D + 16) * 2^-24 of the
two values that a rotation combines."""
import pytest
import torch

import block_wise_fp8_gb300 as fb

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def table(P, rot, base=10000.0):
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / max(rot, 1))
    ang = torch.arange(P, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def reference(v, gamma, tab, pos, eps, inter):
    """(result, bound on its error), both 64 bits."""
    rot, D = tab.shape[1], v.shape[2]
    v = v.double()
    if gamma is not None:
        v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps) * gamma.double()
    ok = (pos >= 0) & (pos < tab.shape[0])
    cs = tab[pos.clamp(0, tab.shape[0] - 1).long()].double()[:, None, :]
    c, s = cs[..., :rot // 2], cs[..., rot // 2:]
    i = torch.arange(rot // 2, device="cuda")
    ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    y, size = v.clone(), v.abs()
    a, b = v[..., ia], v[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    y, size = [torch.where(ok[:, None, None], z, 0.0) for z in (y, size)]
    return y, y.abs() * 2.0 ** -8 + size * (D + 16) * 2.0 ** -24 + 1e-38


def check(y, ref, bound):
    err = (y.double() - ref).abs()
    assert bool((err <= bound).all()), float((err / bound.clamp(min=1e-30)).max())


@pytest.mark.parametrize("T,HQ,HK,D,rot,inter", [
    (1, 1, 1, 16, 16, False), (1, 64, 8, 128, 128, False), (3, 5, 1, 64, 64, True),
    (7, 16, 2, 80, 80, False), (33, 24, 3, 192, 64, False), (33, 24, 3, 192, 64, True),
    (257, 8, 8, 256, 128, False), (5, 3, 2, 512, 512, True), (5, 3, 2, 512, 96, False),
    (2, 4, 4, 96, 0, False), (1021, 7, 1, 48, 32, False)])
def test_norm_and_rotation(T, HQ, HK, D, rot, inter):
    g = torch.Generator("cuda").manual_seed(T * 1000 + D)
    qkv = (torch.randn(T, (HQ + 2 * HK) * D, generator=g, device="cuda") * 3).to(BF16)
    q = qkv[:, :HQ * D].view(T, HQ, D)
    k = qkv[:, HQ * D:(HQ + HK) * D].view(T, HK, D)
    gq = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(BF16)
    gk = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(BF16)
    tab = table(4096, rot)
    pos = torch.randint(0, 4096, (T,), generator=g, device="cuda")
    for gammas, dt in (((gq, gk), torch.int64), ((None, gk), torch.int32), ((None, None), torch.int64)):
        qo, ko = torch.full_like(q, 9.0), torch.full_like(k, 9.0)
        fb.fp8bq_qk_norm_rope(q, k, gammas[0], gammas[1], tab, pos.to(dt), qo, ko, eps=1e-5,
                              interleaved=inter)
        check(qo, *reference(q, gammas[0], tab, pos, 1e-5, inter))
        check(ko, *reference(k, gammas[1], tab, pos, 1e-5, inter))


def test_in_place_on_the_packed_rows_leaves_values_alone():
    g = torch.Generator("cuda").manual_seed(3)
    T, HQ, HK, D = 19, 6, 2, 128
    qkv = torch.randn(T, (HQ + 2 * HK) * D + 64, generator=g, device="cuda").to(BF16)
    was = qkv.clone()
    q = qkv[:, :HQ * D].view(T, HQ, D)
    k = qkv[:, HQ * D:(HQ + HK) * D].view(T, HK, D)
    gam = torch.ones(D, device="cuda", dtype=BF16)
    tab, pos = table(64, D), torch.arange(T, device="cuda")
    rq = reference(was[:, :HQ * D].view(T, HQ, D), gam, tab, pos, 1e-6, False)
    rk = reference(was[:, HQ * D:(HQ + HK) * D].view(T, HK, D), gam, tab, pos, 1e-6, False)
    fb.fp8bq_qk_norm_rope(q, k, gam, gam, tab, pos, q, k)
    check(q, *rq)
    check(k, *rk)
    assert torch.equal(qkv[:, (HQ + HK) * D:], was[:, (HQ + HK) * D:])


def test_head_stride_other_than_the_head_size_and_heads_first():
    g = torch.Generator("cuda").manual_seed(4)
    T, H, D = 9, 5, 64
    q = torch.randn(H, T, D, generator=g, device="cuda").to(BF16).transpose(0, 1)  # heads first
    k = torch.randn(T, H, D + 16, generator=g, device="cuda").to(BF16)[..., :D]
    qo = torch.empty(T, H, D + 8, device="cuda", dtype=BF16)[..., :D]
    ko = torch.empty(H, T, D, device="cuda", dtype=BF16).transpose(0, 1)
    tab, pos = table(32, D), torch.arange(T, device="cuda", dtype=torch.int32)
    fb.fp8bq_qk_norm_rope(q, k, None, None, tab, pos, qo, ko)
    check(qo, *reference(q, None, tab, pos, 0, False))
    check(ko, *reference(k, None, tab, pos, 0, False))


def test_positions_outside_the_table_are_padding():
    T, H, D = 6, 3, 128
    q = torch.ones(T, H, D, device="cuda", dtype=BF16)
    tab = table(16, D)
    pos = torch.tensor([0, -1, 15, 16, 2 ** 40, -2 ** 40], device="cuda")
    out = torch.full_like(q, 7.0)
    fb.fp8bq_qk_norm_rope(q, None, None, None, tab, pos, out, None)
    assert bool((out[[1, 3, 4, 5]] == 0).all())
    check(out, *reference(q, None, tab, pos, 0, False))


def test_zero_and_nonfinite_heads():
    D = 128
    q = torch.zeros(1, 3, D, device="cuda", dtype=BF16)
    q[0, 1, 5] = float("inf")
    q[0, 2, 5] = float("nan")
    out, gam = torch.empty_like(q), torch.ones(D, device="cuda", dtype=BF16)
    tab, pos = table(4, D), torch.ones(1, device="cuda", dtype=torch.int64)
    fb.fp8bq_qk_norm_rope(q, None, gam, None, tab, pos, out, None, eps=1e-6)
    assert bool((out[0, 0] == 0).all())
    assert bool(out[0, 1, 5].isnan()) and bool(out[0, 2].isnan().all())


def test_no_tokens():
    e = torch.empty(0, 4, 64, device="cuda", dtype=BF16)
    fb.fp8bq_qk_norm_rope(e, e, None, None, table(4, 64),
                          torch.empty(0, device="cuda", dtype=torch.int64), e, e)


def test_outputs_of_any_strides_whose_heads_do_not_overlap():
    g = torch.Generator("cuda").manual_seed(5)
    T, H, D = 3, 2, 64
    # one row for all heads and tokens as input; outputs with heads among the tokens
    q = torch.randn(1, 1, D, generator=g, device="cuda").to(BF16).expand(T, H, D)
    tab, pos = table(32, D), torch.arange(T, device="cuda")
    ref = reference(q, None, tab, pos, 0, False)
    for ts, hs in ((2 * D, 3 * D), (3 * D, 2 * D), (D, 3 * D), (D + 8, 4 * D), (2 * D, D)):
        buf = torch.full((10 * D,), 7.0, device="cuda", dtype=BF16)
        out = buf.as_strided((T, H, D), (ts, hs, 1))
        fb.fp8bq_qk_norm_rope(q, None, None, None, tab, pos, out, None)
        check(out, *ref)
        assert int((buf == 7.0).sum()) == 4 * D    # nothing beside the heads
    one = torch.empty(1, H, D, device="cuda", dtype=BF16).expand(T, H, D)
    for out in (one, torch.empty(T, 1, D, device="cuda", dtype=BF16).expand(T, H, D),
                torch.empty(8 * D, device="cuda", dtype=BF16).as_strided((T, H, D), (D, D, 1))):
        with pytest.raises(fb.Fp8bqError, match="ERR_SHAPE"):
            fb.fp8bq_qk_norm_rope(q, None, None, None, tab, pos, out, None)
        with pytest.raises(fb.Fp8bqError, match="ERR_SHAPE"):
            fb.fp8bq_qk_norm_rope(q, q, None, None, tab, pos, torch.empty_like(q.contiguous()), out)
    # one token's expanded token stride means nothing
    out = torch.empty(1, H, D, device="cuda", dtype=BF16)
    fb.fp8bq_qk_norm_rope(q[:1], None, None, None, tab, pos[:1], out.as_strided((1, H, D), (0, D, 1)), None)
    check(out, ref[0][:1], ref[1][:1])


@pytest.mark.parametrize("name", ["q_gamma", "table", "positions", "q_out", "k_out"])
@pytest.mark.parametrize("value", [[1.0], None, 5])
def test_what_is_no_tensor_is_refused(name, value):
    T, H, D = 3, 2, 64
    q = torch.ones(T, H, D, device="cuda", dtype=BF16)
    d = dict(q=q, k=q.clone(), q_gamma=None, k_gamma=None, table=table(8, D),
             positions=torch.zeros(T, device="cuda", dtype=torch.int32), q_out=q.clone(), k_out=q.clone())
    if name == "q_gamma" and value is None:
        return
    d[name] = value
    with pytest.raises(ValueError):
        fb.fp8bq_qk_norm_rope(*d.values())
