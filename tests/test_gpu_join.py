"""GPU parity of the MXFP4 quantiser and of what stands between two blocks with the float64
definitions in oracle/block4.py. Tolerances count roundings, as in test_gpu_dense.py."""
import numpy as np
import pytest
import torch

from oracle import bf16_bits_from_f32, bf16_round_f64, block4, dense
from gpu_helpers import to_dev
from test_gpu_dense import (BF, F32, NORM_SHAPES, U32, UBF, draw, norm_bound, out_t, rng, ueps, val,
                            within)

pytestmark = pytest.mark.gpu
moe4 = pytest.importorskip("bit_mixture_experts_amd.moe4")


# ------------------------------------------------------------------- MXFP4

def quantize_check(t):
    sh = tuple(t.shape)
    nb = sh[:-1] + (sh[-1] // 32,)
    q, s, v = out_t(nb + (16,), torch.uint8), out_t(nb, torch.uint8), out_t(sh, BF)
    moe4.moe4_quantize_mxfp4(t, q.t, s.t, values=v.t)
    wq, ws = block4.quantize_mxfp4(val(t))
    assert np.array_equal(s.t.cpu().numpy(), ws)
    assert np.array_equal(q.t.cpu().numpy(), wq)
    wv, gv = block4.values_mxfp4(wq, ws), val(v.t)
    assert np.array_equal(np.isnan(gv), np.isnan(wv))
    # a largest value above 3.5 * 2^126 takes code 4 of scale 2^126: 2^128, past bf16's range
    wv = np.where(np.abs(wv) >= 2.0 ** 128, np.copysign(np.inf, wv), wv)
    assert np.array_equal(gv[~np.isnan(wv)], wv[~np.isnan(wv)])
    # the codes alone are the same
    q2, s2 = torch.zeros_like(q.t), torch.zeros_like(s.t)
    moe4.moe4_quantize_mxfp4(t, q2, s2)
    assert torch.equal(q2, q.t) and torch.equal(s2, s.t)
    for g in (q, s, v):
        g.check("quantize")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R,K", [(1, 32), (3, 64), (7, 96), (5, 2880), (129, 1056), (1, 65536)])
def test_quantize_mxfp4_bit_exact(R, K, dtype):
    r = rng("mx4", R, K)
    x = (r.standard_normal((R, K)) * np.exp2(r.integers(-30, 30, (R, K // 32))).repeat(32, 1)).astype(np.float32)
    x.reshape(-1)[:8] = [0.0, -0.0, 6.0, 7.0, 0.25, 0.75, -2.5, 5.0]
    if R > 2:
        x[1, :32] = 0.0
        x[2, 5], x[2, 40] = np.inf, np.nan
        x[0, 32:64] = 1e-45      # fp32 subnormals
        x[1, 32:64] = np.ldexp(r.standard_normal(32), -124).astype(np.float32)
    if R > 4:
        x[4, :32] = (r.standard_normal(32) * 1e38).astype(np.float32)   # the largest scales
        x[4, 33] = 3.3e38
    quantize_check(to_dev(bf16_bits_from_f32(x)) if dtype == BF else to_dev(x))


@pytest.mark.parametrize("exp", [-126, -100, 0, 1, 60, 124])
def test_quantize_mxfp4_every_rounding(exp):
    # every value, every midpoint and the floats next to each, both signs, at several scales
    m = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], np.float32)
    mid = ((m[:-1] + m[1:]) / 2).astype(np.float32)
    v = np.concatenate([m, mid, np.nextafter(mid, np.float32(9)), np.nextafter(mid, np.float32(0))])
    for top in (6.0, 7.0, np.nextafter(np.float32(7), np.float32(9)), 4.0):
        x = np.zeros((2, 32), np.float32)
        x[:, 0] = top
        x[0, 1:1 + len(v)], x[1, 1:1 + len(v)] = v, -v
        quantize_check(to_dev(np.ldexp(x, exp).astype(np.float32)))


def test_quantize_mxfp4_in_place_and_shapes():
    r = rng("mx4-shape")
    x, _ = draw(r, (2, 3, 64))
    q = torch.empty((2, 3, 2, 16), dtype=torch.uint8, device="cuda")
    s = torch.empty((2, 3, 2), dtype=torch.float8_e8m0fnu, device="cuda")
    v = torch.empty_like(x)
    moe4.moe4_quantize_mxfp4(x, q, s, values=v)
    keep = x.clone()
    moe4.moe4_quantize_mxfp4(x, q, s, values=x)
    assert torch.equal(x, v)
    # what was rounded once stays: codes stand for themselves
    q2, s2, v2 = torch.empty_like(q), torch.empty_like(s), torch.empty_like(v)
    moe4.moe4_quantize_mxfp4(v, q2, s2, values=v2)
    assert torch.equal(v2, v)
    dec = torch.empty_like(x)
    moe4.moe4_decode_mxfp4(q, s.view(torch.uint8), dec)
    assert torch.equal(dec, v)
    for bad in ((x[..., :33].contiguous(), q, s), (x, q[:1], s), (x, q, s[..., :1].contiguous())):
        with pytest.raises((ValueError, moe4.Moe4Error)):
            moe4.moe4_quantize_mxfp4(*bad)
    assert keep.shape == x.shape
    moe4.moe4_quantize_mxfp4(x[:0], q[:0], s[:0])


# -------------------------------------------------------------------- join

RS, BS = 0.8125, 1.625
ROUND = {BF: bf16_round_f64, F32: None}


@pytest.mark.parametrize("bd,sd,post,pre,gated,res", [
    (BF, BF, True, True, True, True), (F32, BF, True, True, False, True), (BF, F32, True, True, True, True),
    (F32, F32, False, True, True, True), (BF, BF, False, True, False, False), (BF, BF, True, False, True, True)])
@pytest.mark.parametrize("T,H", NORM_SHAPES)
def test_join_norm(T, H, bd, sd, post, pre, gated, res):
    r = rng("join", T, H)
    wd = BF if bd == BF else F32
    b, bv = draw(r, (T, H), bd, 3.0)
    rs, rv = draw(r, (T, H), sd, 2.0) if res else (None, None)
    wo, wov = draw(r, (H,), wd) if post else (None, None)
    wi, wiv = draw(r, (H,), F32 if wd == BF else BF) if pre else (None, None)
    gate, gv = draw(r, (T,), F32) if gated else (None, None)
    if T > 1:   # a row of zeros
        b[1], bv[1] = 0, 0
        if res:
            rs[1], rv[1] = 0, 0
    so = out_t((T, H), sd)
    ro, ri = out_t((T,), F32) if post else None, out_t((T,), F32) if pre else None
    out = out_t((T, H), BF) if pre else None
    low = pre and H % 32 == 0
    q8 = (out_t((T, H), torch.uint8), out_t((T, H // 32), torch.uint8)) if low else (None, None)
    q4 = (out_t((T, H // 32, 16), torch.uint8), out_t((T, H // 32), torch.uint8)) if low else (None, None)
    t = lambda g: g.t if g else None   # noqa: E731
    for q in (q8, q4):
        moe4.moe4_join_norm(b, wi, 1e-6, residual=rs, res_scale=RS, block_scale=BS, gate=gate, w_post=wo,
                            sum_out=so.t, out=t(out), out_q=t(q[0]), out_s=t(q[1]), rstd_post=t(ro),
                            rstd_pre=t(ri))
    e = norm_bound(H)
    f = block4.join_norm(bv, rv, RS, BS, gv, wov, None, 1e-6)
    if post:
        within(ro.t.double().cpu().numpy(), f["ro"], e * f["ro"], "rstd_post")
    # the sum: rstd's error and five roundings of the block's term, one of each term, and the sum's own
    block = np.abs(f["s"] - (RS * rv if res else 0))
    within(val(so.t), f["s"], ueps(sd) * np.abs(f["s"]) + (e + 8 * U32) * block
           + (2 * U32 * RS * np.abs(rv) if res else 0) + 1e-38, "sum")
    if pre:
        # the second norm on the row that the stream holds
        s = val(so.t)
        wr = 1 / np.sqrt(np.mean(s * s, 1) + 1e-6)
        wy = s * wr[:, None] * wiv
        within(ri.t.double().cpu().numpy(), wr, e * wr, "rstd_pre")
        within(val(out.t), wy, (UBF + 2 * e) * np.abs(wy) + 1e-38, "out")
    if low:
        g8 = dense.mxfp8_values(q8[0].t.cpu().numpy(), q8[1].t.cpu().numpy())
        g4 = block4.values_mxfp4(q4[0].t.cpu().numpy(), q4[1].t.cpu().numpy())
        for got, sc, (wq, ws), half, floor, what in (
                (g8, q8[1], dense.quantize_mxfp8(wy), 2.0 ** -4, 2.0 ** -9, "MXFP8"),
                (g4, q4[1], block4.quantize_mxfp4(wy), 0.25, 0.25, "MXFP4")):
            # half a step of the code plus the fp32 error; a block within that error of a power of
            # two may take the neighbouring scale (whose step at the bottom is twice as large)
            d = np.abs(ws.astype(int) - sc.t.cpu().numpy().astype(int))
            assert d.max() <= 1 and np.mean(d > 0) <= 1e-3
            scale = np.ldexp(1.0, np.maximum(ws, sc.t.cpu().numpy()).astype(int) - 127).repeat(32, 1)
            within(got, wy, (half + 2 * e) * np.abs(wy) + floor * scale + 1e-38, what)
        for g in (*q8, *q4):
            g.check("codes")
    for g in (so, ro, ri, out):
        if g is not None:
            g.check("join")


def test_join_norm_is_add_rmsnorm_where_they_meet():
    r = rng("join-add")
    b, _ = draw(r, (33, 1056))
    rs, _ = draw(r, (33, 1056))
    w, _ = draw(r, (1056,))
    outs = [torch.empty_like(b) for _ in range(4)]
    moe4.moe4_add_rmsnorm(b, w, 1e-6, residual=rs, sum_out=outs[0], out=outs[1])
    moe4.moe4_join_norm(b, w, 1e-6, residual=rs, sum_out=outs[2], out=outs[3])
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
    # in place: the stream, or the block's output, takes the sum
    for where in (0, 1):
        a, c = b.clone(), rs.clone()
        moe4.moe4_join_norm(a, w, 1e-6, residual=c, sum_out=(c, a)[where], out=outs[3])
        assert torch.equal((c, a)[where], outs[2]) and torch.equal(outs[1], outs[3])


def test_join_norm_non_finite_rows_stay_apart():
    r = rng("join-nan")
    b, _ = draw(r, (5, 96))
    rs, _ = draw(r, (5, 96))
    w, _ = draw(r, (96,))
    b[1, 7], rs[2, 95], b[3, 0] = float("nan"), float("inf"), float("inf")
    s, out = torch.empty_like(b), torch.empty_like(b)
    q = torch.empty((5, 3, 16), dtype=torch.uint8, device="cuda")
    qs = torch.empty((5, 3), dtype=torch.uint8, device="cuda")
    moe4.moe4_join_norm(b, w, 1e-6, residual=rs, w_post=w, sum_out=s, out=out, out_q=q, out_s=qs)
    o = val(out)
    assert np.isnan(o[1]).all() and np.isnan(o[2, 95]) and np.isfinite(o[[0, 4]]).all()
    assert np.isnan(o[3]).all()      # inf * rstd 0
    assert (qs.cpu().numpy()[[1, 3]] == 255).all() and (qs.cpu().numpy()[[0, 4]] != 255).all()
    assert (q.cpu().numpy()[1] == 0).all()


@pytest.mark.parametrize("yd,sd,bd,post,pre,gated,past", [
    (BF, BF, BF, True, True, True, True), (F32, BF, F32, True, True, False, True),
    (BF, F32, BF, False, True, True, False), (F32, F32, F32, True, True, True, False),
    (BF, BF, BF, True, False, True, True), (BF, F32, F32, False, False, False, True)])
@pytest.mark.parametrize("T,H", NORM_SHAPES)
def test_join_norm_backward(T, H, yd, sd, bd, post, pre, gated, past):
    r = rng("join-bwd", T, H)
    wd = BF if bd == BF else F32
    dy, yv = draw(r, (T, H), yd, 0.1)
    s, sv = draw(r, (T, H), sd, 1.5)
    b, bv = draw(r, (T, H), bd, 3.0)
    ds, ev = draw(r, (T, H), sd, 0.1) if past or not pre else (None, None)
    wo, wov = draw(r, (H,), wd) if post else (None, None)
    wi, wiv = draw(r, (H,), wd) if pre else (None, None)
    gate, gv = draw(r, (T,), F32) if gated else (None, None)

    def rstd(v):
        t = to_dev((1 / np.sqrt(np.mean(v * v, 1) + 1e-6)).astype(np.float32))
        return t, t.double().cpu().numpy()
    ro, rov = rstd(bv) if post else (None, None)
    ri, riv = rstd(sv) if pre else (None, None)
    ws = torch.full((moe4.moe4_join_norm_workspace_size(T, H),), 0xFF, dtype=torch.uint8, device="cuda")
    db, dres = out_t((T, H), bd), out_t((T, H), sd)
    dg = out_t((T,), F32) if gated else None
    dwo, dwi = out_t((H,), F32) if post else None, out_t((H,), F32) if pre else None
    t = lambda g: g.t if g else None   # noqa: E731
    args = (dy if pre else None, s if pre else None, b, wi, ri)
    kw = dict(ds=ds, res_scale=RS, block_scale=BS, gate=gate, w_post=wo, rstd_post=ro)
    moe4.moe4_join_norm_backward(*args, db.t, dres=dres.t, dgate=t(dg), dw_post=t(dwo), dw_pre=t(dwi),
                                 ws=ws, **kw)
    w = block4.join_norm_backward(yv, sv, bv, ev, RS, BS, gv, wov, wiv, rov, riv)
    # magnitudes that the roundings act on: of dS, then of what is made of it
    e = (min(H, 512) + 24) * U32
    mS = np.zeros((T, H)) if ev is None else np.abs(ev)
    if pre:
        n, p = np.abs(sv * riv[:, None]), np.abs(yv * wiv)
        mS = mS + riv[:, None] * (p + n * np.mean(p * n, 1, keepdims=True))
    within(val(dres.t), w["dres"], ueps(sd) * np.abs(w["dres"]) + e * RS * mS + 1e-38, "dres")
    c = BS * (np.abs(gv) if gated else np.ones(T))
    m = np.abs(bv * rov[:, None]) if post else np.abs(bv)
    q = mS * np.abs(wov) if post else mS
    if post:
        mb = c[:, None] * rov[:, None] * (q + m * np.mean(q * m, 1, keepdims=True))
    else:
        mb = c[:, None] * mS
    within(val(db.t), w["db"], ueps(bd) * np.abs(w["db"]) + 2 * e * mb + 1e-38, "db")
    if gated:
        within(dg.t.double().cpu().numpy(), w["dgate"], 2 * e * BS * np.sum(q * m, 1) + 1e-38, "dgate")
    if post:
        # T terms of a column, each with dS's own error
        within(dwo.t.double().cpu().numpy(), w["dw_post"],
               ((T + 8) * U32 + e) * np.sum(c[:, None] * mS * m, 0) + 1e-38, "dw_post")
    if pre:
        within(dwi.t.double().cpu().numpy(), w["dw_pre"],
               (T + 8) * U32 * np.sum(np.abs(yv * sv * riv[:, None]), 0) + 1e-38, "dw_pre")
    for g in (db, dres, dg, dwo, dwi):
        if g is not None:
            g.check("backward")
    # one output at a time, and in place, the same bits
    d2 = b.clone()
    moe4.moe4_join_norm_backward(args[0], args[1], d2, *args[3:], d2, **kw)
    assert torch.equal(d2, db.t)
    if post and pre:
        for name, full in (("dw_post", dwo), ("dw_pre", dwi)):
            one = out_t((H,), F32)
            moe4.moe4_join_norm_backward(*args, d2, ws=ws, **{name: one.t}, **kw)
            assert torch.equal(one.t, full.t)
    if ds is not None:
        d3 = ds.clone()
        kw["ds"] = d3
        moe4.moe4_join_norm_backward(*args, d2, dres=d3, **kw)
        assert torch.equal(d3, dres.t)


def test_join_norm_backward_against_differences():
    r = rng("join-diff")
    T, H = 6, 160
    b, bv = draw(r, (T, H), F32)
    rs, rv = draw(r, (T, H), F32)
    wo, wov = draw(r, (H,), F32)
    wi, wiv = draw(r, (H,), F32)
    gate, gv = draw(r, (T,), F32)
    dy, yv = draw(r, (T, H), F32)
    ds, ev = draw(r, (T, H), F32)
    s, out = torch.empty_like(b), torch.empty((T, H), dtype=BF, device="cuda")
    ro, ri = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    moe4.moe4_join_norm(b, wi, 1e-5, residual=rs, res_scale=RS, block_scale=BS, gate=gate, w_post=wo,
                        sum_out=s, out=out, rstd_post=ro, rstd_pre=ri)
    g = {k: torch.empty_like(v) for k, v in dict(db=b, dres=b, dgate=gate, dw_post=wo, dw_pre=wi).items()}
    ws = torch.empty(moe4.moe4_join_norm_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    moe4.moe4_join_norm_backward(dy, s, b, wi, ri, ds=ds, res_scale=RS, block_scale=BS, gate=gate, w_post=wo,
                                 rstd_post=ro, ws=ws, **g)
    v = dict(b=bv, residual=rv, gate=gv, w_post=wov, w_pre=wiv)

    def loss(**over):
        f = block4.join_norm(**{**v, **over}, res_scale=RS, block_scale=BS, eps=1e-5)
        return np.sum(f["s"] * ev) + np.sum(f["y"] * yv)
    for name, key in (("b", "db"), ("residual", "dres"), ("gate", "dgate"), ("w_post", "dw_post"),
                      ("w_pre", "dw_pre")):
        u, h = r.standard_normal(v[name].shape), 1e-5
        want = (loss(**{name: v[name] + h * u}) - loss(**{name: v[name] - h * u})) / (2 * h)
        got = g[key].double().cpu().numpy()
        assert abs(np.sum(got * u) - want) <= 1e-5 * np.sum(np.abs(got * u)), key


def test_join_norm_no_rows_and_refusals():
    H = 64
    e = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype, device="cuda")   # noqa: E731
    w = e(H)
    moe4.moe4_join_norm(e(0, H), w, 1e-6, residual=e(0, H), sum_out=e(0, H), out=e(0, H))
    dw = torch.full((H,), 7.0, device="cuda")
    moe4.moe4_join_norm_backward(e(0, H), e(0, H), e(0, H), w, e(0, dtype=F32), e(0, H), dw_pre=dw)
    assert bool((dw == 0).all())
    b, ok = e(2, H), dict(residual=e(2, H), sum_out=e(2, H), out=e(2, H))
    for kw, err in ((dict(residual=e(2, H, dtype=F32)), TypeError), (dict(residual=e(3, H)), ValueError),
                    (dict(gate=e(3, dtype=F32)), ValueError), (dict(gate=e(2)), TypeError),
                    (dict(w_post=e(H + 8)), ValueError), (dict(out=e(2, H, dtype=F32)), TypeError),
                    (dict(rstd_post=e(2, dtype=F32)), moe4.Moe4Error),
                    (dict(out_q=e(2, H, dtype=torch.uint8)), moe4.Moe4Error),
                    (dict(out_q=e(2, 2, 15, dtype=torch.uint8), out_s=e(2, 2, dtype=torch.uint8)), ValueError),
                    (dict(residual=torch.zeros(2, H, dtype=BF)), TypeError)):
        with pytest.raises(err):
            moe4.moe4_join_norm(b, w, 1e-6, **{**ok, **kw})
    with pytest.raises(moe4.Moe4Error):
        moe4.moe4_join_norm(b, None, 1e-6, **ok)          # y without its norm
    r = e(2, dtype=F32)
    for a, kw, err in (((b, b, b, w, r, e(2, H, dtype=F32)), {}, TypeError), ((b, b, b, w, r, b), dict(dres=b), moe4.Moe4Error),
                       ((b, b, b, w, r, b), dict(dw_post=e(H, dtype=F32)), moe4.Moe4Error),
                       ((b, b, b, w, r, b), dict(dw_pre=e(H, dtype=F32)), moe4.Moe4Error),   # no workspace
                       ((b, b, b, w, r, b), dict(w_post=w), moe4.Moe4Error),
                       ((None, None, b, None, None, b), {}, moe4.Moe4Error)):
        with pytest.raises(err):
            moe4.moe4_join_norm_backward(*a, **kw)


def test_join_offsets_past_32_bits():
    # tensors of more than 2^32 bytes: the last rows are those of a call on them alone
    H, T, tail = 2048, 1_060_000, 300
    gen = torch.Generator(device="cuda").manual_seed(6)
    b = torch.randn((T, H), generator=gen, device="cuda", dtype=BF)
    res = torch.randn((T, H), generator=gen, device="cuda", dtype=BF)
    w = torch.ones(H, device="cuda", dtype=BF)
    e = lambda n, *s, dtype=BF: torch.empty((n, *s), dtype=dtype, device="cuda")   # noqa: E731

    def run(b, res, n):
        s, q, qs = e(n, H), e(n, H // 32, 16, dtype=torch.uint8), e(n, H // 32, dtype=torch.uint8)
        ro, ri = e(n, dtype=F32), e(n, dtype=F32)
        moe4.moe4_join_norm(b, w, 1e-6, residual=res, w_post=w, sum_out=s, out_q=q, out_s=qs, rstd_post=ro, rstd_pre=ri)
        return s, q, qs, ro, ri
    big, small = run(b, res, T), run(b[-tail:].clone(), res[-tail:].clone(), tail)
    # (another number of rows takes another split of the row's sum: c = rstd differs by few steps of
    # 2^-24 of H terms, s by that and, where it falls at a border, by one bf16 step)
    assert torch.allclose(big[3][-tail:], small[3], rtol=2 * (H + 8) * U32, atol=0)
    assert torch.allclose(big[0][-tail:].float(), small[0].float(), rtol=2.0 ** -7, atol=1e-4)
    assert (big[1][-tail:] != small[1]).float().mean() < 1e-2 and (big[2][-tail:] != small[2]).float().mean() < 1e-2
    x = big[0]
    q, qs = e(T, H // 32, 16, dtype=torch.uint8), e(T, H // 32, dtype=torch.uint8)
    moe4.moe4_quantize_mxfp4(x, q, qs)
    q2, s2 = e(tail, H // 32, 16, dtype=torch.uint8), e(tail, H // 32, dtype=torch.uint8)
    moe4.moe4_quantize_mxfp4(x[-tail:].clone(), q2, s2)
    assert torch.equal(q[-tail:], q2) and torch.equal(qs[-tail:], s2)
    db, dres = torch.empty_like(b), torch.empty_like(b)
    kw = dict(w_post=w)
    moe4.moe4_join_norm_backward(res, x, b, w, big[4], db, dres=dres, rstd_post=big[3], **kw)
    d2, r2 = e(tail, H), e(tail, H)
    moe4.moe4_join_norm_backward(res[-tail:].clone(), x[-tail:].clone(), b[-tail:].clone(), w, big[4][-tail:].clone(), d2,
                                 dres=r2, rstd_post=big[3][-tail:].clone(), **kw)
    # rows are independent of each other; the sums' split may differ, by 2 (H + 8) 2^-24 of the terms'
    # magnitudes (of order one here), and a rounding to bf16 then by a step
    for a, c in ((db, d2), (dres, r2)):
        assert torch.allclose(a[-tail:].float(), c.float(), rtol=2.0 ** -7, atol=1e-3)
