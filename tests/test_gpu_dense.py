"""GPU parity of the dense operators with the float64 definitions in oracle/dense.py.

Tolerances count roundings: half a step of bf16 is 2^-8 of the value, of fp32 2^-24, of e4m3
2^-4. A sum of n fp32 terms is off by at most n 2^-24 times the sum of their magnitudes,
whatever the order. Where a product's operand is rounded to bf16 the errors of its many terms
are independent, and each is at most 2^-8 / sqrt(3) of its value in the root mean square, so a
whole row of outputs is held in the 2-norm too: r roundings on the way, and a factor of two for
the spread of one row."""
import math
import zlib

import numpy as np
import pytest
import torch

from oracle import bf16_bits_from_f32, bf16_bits_to_f64, bf16_round_f64, dense
from gpu_helpers import DEV, bits, f64, say, to_dev

pytestmark = pytest.mark.gpu
moe4 = pytest.importorskip("bit_mixture_experts_amd.moe4")

U32, UBF = 2.0 ** -24, 2.0 ** -8
RMS_BF = UBF / math.sqrt(3)
BF, F32 = torch.bfloat16, torch.float32


def rng(*key):
    return np.random.default_rng([zlib.crc32(k.encode()) if isinstance(k, str) else int(k) for k in key])


def draw(r, shape, dtype=BF, std=1.0):
    """(device tensor, its values in float64)"""
    a = (r.standard_normal(shape) * std).astype(np.float32)
    if dtype == BF:
        b = bf16_bits_from_f32(a)
        return to_dev(b), bf16_bits_to_f64(b)
    return to_dev(a), a.astype(np.float64)


def val(t):
    return f64(t) if t.dtype == BF else t.double().cpu().numpy()


def ueps(dtype):
    return UBF if dtype == BF else U32


class Guarded:
    """An output tensor between two bands of sentinels that no kernel may touch."""

    def __init__(self, shape, dtype, fill=None):
        n = int(np.prod(shape))
        self.n, self.dtype = n, dtype
        self.raw = torch.full((n * torch.empty(0, dtype=dtype).element_size() + 1024,), 0xA5,
                              dtype=torch.uint8, device="cuda")
        self.t = self.raw[512:512 + n * torch.empty(0, dtype=dtype).element_size()].view(dtype).view(shape)

    def check(self, what):
        assert bool((self.raw[:512] == 0xA5).all()) and bool((self.raw[-512:] == 0xA5).all()), \
            f"{what}: written outside its bounds"


def out_t(shape, dtype):
    return Guarded(tuple(shape), dtype)


def within(got, want, tol, what):
    err = np.abs(got - want)
    worst = float(np.max(err - tol)) if err.size else 0.0
    say(f"  {what}: max|err| {float(err.max()) if err.size else 0:.3e}, "
        f"worst share of the bound {float(np.max(err / np.maximum(tol, 1e-300))) if err.size else 0:.3f}")
    assert worst <= 0, f"{what}: {worst} beyond the bound"


# ------------------------------------------------------------------- MXFP8

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R,K", [(1, 32), (3, 64), (7, 96), (5, 2880), (129, 1056), (1, 65536)])
def test_quantize_mxfp8_bit_exact(R, K, dtype):
    r = rng("mx", R, K)
    x = (r.standard_normal((R, K)) * np.exp2(r.integers(-30, 30, (R, K // 32))).repeat(32, 1)).astype(np.float32)
    x.reshape(-1)[:8] = [0.0, -0.0, 448.0, 464.0, 2.0 ** -9, 2.0 ** -10, -3 * 2.0 ** -10, 480.0]
    if R > 2:
        x[1, :32] = 0.0
        x[2, 5], x[2, 40] = np.inf, np.nan
        x[0, 32:64] = 1e-45      # fp32 subnormals
    t = to_dev(bf16_bits_from_f32(x)) if dtype == BF else to_dev(x)
    q, s = out_t((R, K), torch.uint8), out_t((R, K // 32), torch.uint8)
    moe4.moe4_quantize_mxfp8(t, q.t, s.t)
    wq, ws = dense.quantize_mxfp8(val(t))
    assert np.array_equal(s.t.cpu().numpy(), ws)
    assert np.array_equal(q.t.cpu().numpy(), wq)
    q.check("q"), s.check("s")


def test_quantize_mxfp8_every_rounding():
    # every e4m3 value, every midpoint between neighbours and the floats next to each, exactly
    t = dense.mxfp8_values(np.arange(127, dtype=np.uint8).repeat(32)[:127 * 32], np.full(127, 127, np.uint8))
    t = t[::32].astype(np.float32)
    mid = ((t[:-1] + t[1:]) / 2).astype(np.float32)
    v = np.concatenate([t, mid, np.nextafter(mid, np.float32(1e9)), np.nextafter(mid, np.float32(0))])
    v = np.concatenate([v, -v])
    x = np.zeros((-(-len(v) // 31), 32), np.float32)
    x[:, 0] = 448.0
    flat = np.zeros(x.shape[0] * 31, np.float32)
    flat[:len(v)] = v
    x[:, 1:] = flat.reshape(-1, 31)
    q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((x.shape[0], 1), dtype=torch.float8_e8m0fnu, device="cuda")
    moe4.moe4_quantize_mxfp8(to_dev(x), q, s)
    wq, ws = dense.quantize_mxfp8(x)
    assert np.array_equal(q.view(torch.uint8).cpu().numpy(), wq)
    assert np.array_equal(s.view(torch.uint8).cpu().numpy(), ws)


# -------------------------------------------------------------------- norm

# every (waves, chunks) instance of the kernels, by rows and columns
NORM_SHAPES = [(1, 8), (3, 64), (1, 2048), (5, 2880), (17, 520), (2, 4096), (3, 8192), (2, 16384),
               (1, 12344), (2050, 1000), (2051, 2048), (2049, 2880), (2048, 4088), (2049, 512), (2048, 64)]


def norm_bound(H):
    """Relative error of rstd in fp32: the sum of at most H squares (of one sign), each rounded,
    the mean, eps, and the root; the lane and wave sums add far fewer terms in a row than H."""
    return (min(H, 512) + 16) * U32


@pytest.mark.parametrize("xd,rd,wd", [(BF, BF, BF), (F32, BF, BF), (BF, F32, F32), (F32, F32, BF),
                                      (BF, None, BF), (F32, None, F32)])
@pytest.mark.parametrize("T,H", NORM_SHAPES)
def test_add_rmsnorm(T, H, xd, rd, wd):
    r = rng("norm", T, H)
    x, xv = draw(r, (T, H), xd)
    w, wv = draw(r, (H,), wd)
    res, rv = draw(r, (T, H), rd, 2.0) if rd is not None else (None, None)
    if T > 1:   # a row of zeros
        x[1] = 0
        xv[1] = 0
        if res is not None:
            res[1] = 0
            rv[1] = 0
    mx = H % 32 == 0
    out, rstd = out_t((T, H), BF), out_t((T,), F32)
    so = out_t((T, H), rd) if rd is not None else None
    q, qs = (out_t((T, H), torch.uint8), out_t((T, H // 32), torch.uint8)) if mx else (None, None)
    moe4.moe4_add_rmsnorm(x, w, 1e-6, residual=res, sum_out=so.t if so else None, out=out.t,
                          out_q=q.t if mx else None, out_s=qs.t if mx else None, rstd=rstd.t)
    # the sum: one fp32 addition, one rounding, on the same values
    if rd is not None:
        want = x.float().cpu() + res.float().cpu()
        want = want.to(rd)
        assert torch.equal(so.t.cpu().view(torch.int16 if rd == BF else torch.int32),
                           want.view(torch.int16 if rd == BF else torch.int32))
        s = want.double().numpy()
    else:
        s = xv
    _, wr, wy = dense.add_rmsnorm(s, wv, 1e-6)
    e = norm_bound(H)
    within(rstd.t.double().cpu().numpy(), wr, e * wr, "rstd")
    within(val(out.t), wy, (UBF + 2 * e) * np.abs(wy) + 1e-38, "out")
    if mx:
        oq, os_ = dense.quantize_mxfp8(wy)
        gv = dense.mxfp8_values(q.t.cpu().numpy(), qs.t.cpu().numpy())
        # half a step of the code (2^-4 of the value, 2^-10 of the scale near zero) plus the
        # fp32 error; a block within that error of a power of two may take the next scale
        scale = np.ldexp(1.0, os_.astype(int) - 127).repeat(32, 1)
        near = np.abs(os_.astype(int) - qs.t.cpu().numpy().astype(int))
        assert near.max() <= 1 and np.mean(near > 0) <= 1e-3
        within(gv, wy, (2.0 ** -4 + 2 * e) * np.abs(wy) + scale * 2.0 ** -9, "MXFP8")
        assert np.mean(q.t.cpu().numpy() != oq) <= 1e-3 + 2.0 / oq.size
        q.check("q"), qs.check("qs")
    for g in (out, rstd, so):
        if g is not None:
            g.check("norm")


def test_add_rmsnorm_in_place_and_alone():
    r = rng("norm-inplace")
    x, _ = draw(r, (9, 512))
    res, _ = draw(r, (9, 512))
    w, _ = draw(r, (512,))
    outs = []
    for where in ("fresh", "res", "x"):
        a, b = x.clone(), res.clone()
        so = {"fresh": torch.empty_like(b), "res": b, "x": a}[where]
        out = torch.empty_like(x)
        moe4.moe4_add_rmsnorm(a, w, 1e-5, residual=b, sum_out=so, out=out)
        outs.append((so, out))
    for so, out in outs[1:]:
        assert torch.equal(so, outs[0][0]) and torch.equal(out, outs[0][1])
    # MXFP8 alone, and the bf16 output alone without a sum, match the call that writes all
    q, qs = torch.empty((9, 512), dtype=torch.uint8, device="cuda"), torch.empty((9, 16), dtype=torch.uint8, device="cuda")
    q2, qs2 = torch.empty_like(q), torch.empty_like(qs)
    out = torch.empty_like(x)
    moe4.moe4_add_rmsnorm(x, w, 1e-5, residual=res, out_q=q, out_s=qs)
    moe4.moe4_add_rmsnorm(x, w, 1e-5, residual=res, out=out, out_q=q2, out_s=qs2)
    assert torch.equal(q, q2) and torch.equal(qs, qs2) and torch.equal(out, outs[0][1])


def test_add_rmsnorm_non_finite_rows_stay_apart():
    r = rng("norm-nan")
    x, xv = draw(r, (4, 96))
    w, wv = draw(r, (96,))
    x[1, 7], x[2, 95] = float("nan"), float("inf")
    out = torch.empty_like(x)
    q, qs = torch.empty((4, 96), dtype=torch.uint8, device="cuda"), torch.empty((4, 3), dtype=torch.uint8, device="cuda")
    moe4.moe4_add_rmsnorm(x, w, 1e-6, out=out, out_q=q, out_s=qs)
    o = val(out)
    assert np.isnan(o[1]).all() and np.isnan(o[2, 95]) and np.isfinite(o[[0, 3]]).all()
    assert (qs.cpu().numpy()[1] == 255).all() and (q.cpu().numpy()[1] == 0x7F).all()
    assert (qs.cpu().numpy()[[0, 3]] != 255).all()


@pytest.mark.parametrize("yd,sd,dd,wd", [(BF, BF, BF, BF), (F32, BF, BF, BF), (BF, F32, F32, F32),
                                         (F32, F32, F32, BF)])
@pytest.mark.parametrize("T,H", NORM_SHAPES)
def test_add_rmsnorm_backward(T, H, yd, sd, dd, wd):
    r = rng("norm-bwd", T, H)
    dy, yv = draw(r, (T, H), yd, 0.1)
    s, sv = draw(r, (T, H), sd, 1.5)
    w, wv = draw(r, (H,), wd)
    dres, ev = draw(r, (T, H), dd, 0.1)
    rstd = 1 / np.sqrt(np.mean(sv * sv, 1) + 1e-6)
    rt = to_dev(rstd.astype(np.float32))
    rstd = rt.double().cpu().numpy()
    ws = torch.empty(moe4.moe4_add_rmsnorm_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    for with_res in (True, False):
        dx, dw = out_t((T, H), dd), out_t((H,), F32)
        moe4.moe4_add_rmsnorm_backward(dy, s, w, rt, dx.t, dres=dres if with_res else None,
                                       dweight=dw.t, ws=ws)
        wx, ww = dense.add_rmsnorm_backward(yv, sv, wv, rstd, ev if with_res else None)
        n = sv * rstd[:, None]
        p = yv * wv
        # the mean's sum (H terms), the products around it, and the rounding of dx
        e = (min(H, 512) + 24) * U32
        mag = rstd[:, None] * (np.abs(p) + np.abs(n) * np.mean(np.abs(p * n), 1, keepdims=True)) + \
            (np.abs(ev) if with_res else 0)
        within(val(dx.t), wx, ueps(dd) * np.abs(wx) + e * mag + 1e-38, "dx")
        within(dw.t.double().cpu().numpy(), ww, (T + 8) * U32 * np.sum(np.abs(yv * n), 0) + 1e-38, "dweight")
        dx.check("dx"), dw.check("dweight")
    # without dweight no workspace is needed, and dx may be dres
    d2 = dres.clone()
    moe4.moe4_add_rmsnorm_backward(dy, s, w, rt, d2, dres=d2)
    first = out_t((T, H), dd)
    moe4.moe4_add_rmsnorm_backward(dy, s, w, rt, first.t, dres=dres, dweight=dw.t, ws=ws)
    assert torch.equal(d2, first.t)


def test_add_rmsnorm_backward_against_differences():
    # the GPU's gradients along a direction against differences of the float64 forward
    r = rng("norm-diff")
    T, H = 6, 160
    s, sv = draw(r, (T, H), F32)
    w, wv = draw(r, (H,), F32)
    dy, yv = draw(r, (T, H), F32)
    _, rstd, _ = dense.add_rmsnorm(sv, wv, 1e-5)
    dx, dw = torch.empty_like(s), torch.empty_like(w)
    ws = torch.empty(moe4.moe4_add_rmsnorm_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    moe4.moe4_add_rmsnorm_backward(dy, s, w, to_dev(rstd.astype(np.float32)), dx, dweight=dw, ws=ws)
    vs, vw, h = r.standard_normal((T, H)), r.standard_normal(H), 1e-5

    def loss(a, b):
        return np.sum(dense.add_rmsnorm(a, b, 1e-5)[2] * yv)
    ds = (loss(sv + h * vs, wv) - loss(sv - h * vs, wv)) / (2 * h)
    dwd = (loss(sv, wv + h * vw) - loss(sv, wv - h * vw)) / (2 * h)
    gx, gw = dx.double().cpu().numpy(), dw.double().cpu().numpy()
    assert abs(np.sum(gx * vs) - ds) <= 1e-5 * np.sum(np.abs(gx * vs))
    assert abs(np.sum(gw * vw) - dwd) <= 1e-5 * np.sum(np.abs(gw * vw))


# ------------------------------------------------------------ feed-forward

ALPHA, LIMIT = 1.702, 7.0


class Block:
    """A dense block's weights on the device and in float64."""

    def __init__(self, key, H, I, mx=False, clamped=False, bias=False):
        r = rng("ffn", key, H, I)
        self.H, self.I, self.mx, self.clamped = H, I, mx, clamped
        self.layout, self.act = ("interleaved", "clamped") if clamped else ("halves", "swiglu")
        wg, self.wg = draw(r, (2 * I, H), std=(2.5 if clamped else 1.0) / math.sqrt(H))
        wd, self.wd = draw(r, (H, I), std=1 / math.sqrt(I))
        bg, self.bg = draw(r, (2 * I,), std=0.3) if bias else (None, None)
        bd, self.bd = draw(r, (H,), std=0.3) if bias else (None, None)
        kw = {}
        if mx:
            qs = []
            for t, name in ((wg, "wg"), (wd, "wd")):
                q, s = dense.quantize_mxfp8(val(t))
                setattr(self, name, dense.mxfp8_values(q, s))
                qs.append((to_dev(q), to_dev(s)))
            (wg, kw["gu_s"]), (wd, kw["dn_s"]) = qs
        self.ffn = moe4.Ffn(
            moe4.MOE4_FFN_MXFP8 if mx else moe4.MOE4_FFN_BF16, wg, wd, H=H, I=I, gu_bias=bg, dn_bias=bd,
            gu_layout=moe4.MOE4_GU_INTERLEAVED if clamped else moe4.MOE4_GU_HALVES,
            act=moe4.MOE4_ACT_SWIGLU_CLAMPED if clamped else moe4.MOE4_ACT_SWIGLU,
            act_alpha=ALPHA, act_limit=LIMIT, **kw)

    def tokens(self, T, key=0):
        r = rng("tok", key, T, self.H)
        x, xv = draw(r, (T, self.H))
        if not self.mx:
            return x, None, xv
        q, s = dense.quantize_mxfp8(xv)
        return to_dev(q), to_dev(s), dense.mxfp8_values(q, s)

    def ws(self, T, backward=False):
        n = moe4.moe4_ffn_workspace_size(self.ffn, T, backward)
        return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")   # NaNs wherever it is read first


def row_norm(got, want, rel, what, floor=1e-30):
    d = np.linalg.norm(got - want, axis=1)
    n = np.linalg.norm(want, axis=1)
    say(f"  {what}: worst row {float(np.max(d / np.maximum(n, floor))):.2e} of {rel:.2e}")
    assert np.all(d <= rel * n + floor), f"{what}: a row is {float(np.max(d / np.maximum(n, floor)))} off"


FFN_CASES = [
    # T, H, I, mx, clamped, bias
    (1, 64, 32, False, False, False), (1, 8, 8, False, False, True), (3, 72, 40, False, True, True),
    (16, 256, 96, False, False, True), (17, 264, 136, False, True, False), (33, 520, 264, False, False, False),
    (64, 136, 72, False, True, True), (65, 128, 128, False, False, True), (127, 520, 392, False, True, True),
    (129, 264, 520, False, False, False), (300, 200, 328, False, True, True), (513, 392, 264, False, False, True),
    (1, 64, 32, True, False, False), (2, 96, 96, True, True, True), (16, 288, 160, True, False, True),
    (31, 224, 96, True, True, True), (64, 160, 416, True, False, False), (66, 96, 32, True, True, True),
    (129, 544, 288, True, True, True), (300, 352, 544, True, False, True), (515, 64, 96, True, True, False),
]
VARIANTS = {"auto": moe4.MOE4_VARIANT_AUTO, "skinny": moe4.MOE4_VARIANT_SKINNY, "tiled": moe4.MOE4_VARIANT_TILED}


def ffn_check(blk, T, variant, out_dtype, res_dtype, save):
    ffn = blk.ffn.with_variant(variant)
    x, xs, xv = blk.tokens(T)
    r = rng("res", T, blk.H)
    res, rv = draw(r, (T, blk.H), res_dtype) if res_dtype is not None else (None, 0.0)
    out = out_t((T, blk.H), out_dtype)
    gu = out_t((T, 2 * blk.I), F32) if save else None
    moe4.moe4_ffn_forward(ffn, x, out.t, x_s=xs, residual=res, save_gu=gu.t if save else None, ws=blk.ws(T))
    want = dense.ffn_forward(xv, blk.wg, blk.wd, blk.layout, blk.act, blk.bg, blk.bd,
                             alpha=ALPHA, limit=LIMIT)
    got = val(out.t)
    assert np.isfinite(got).all()
    out.check("out")
    # pre-activations: fp32 sums of exact products. The e4m3 matrix instruction aligns the 32
    # products of a block to the largest and keeps each to at least 2^-16 of that one.
    unit = 32 * 2.0 ** -16 if blk.mx else 0.0
    if save:
        gu.check("save_gu")
        mag = np.abs(xv) @ np.abs(blk.wg).T + (0 if blk.bg is None else np.abs(blk.bg))
        within(gu.t.double().cpu().numpy(), want["gu"], ((blk.H + 2) * U32 + unit) * mag, "gu")
    # the product without the residual, as a row: h rounded once (bf16) or to e4m3 (half a step
    # of 2^-4, 2^-4 / sqrt(3) in the root mean square), and out rounded once
    rms_h = 2.0 ** -4 / math.sqrt(3) if blk.mx else RMS_BF
    plain = want["out"]
    bound = 2 * (rms_h + 1e-5) * np.linalg.norm(plain, axis=1) + \
        ueps(out_dtype) * np.linalg.norm(plain + rv, axis=1)
    d = np.linalg.norm(got - (plain + rv), axis=1)
    say(f"  out: worst row {float(np.max(d / bound)):.2f} of the bound")
    assert np.all(d <= bound)
    if blk.mx:
        # against the definition with h quantised as the kernel does: only values of h within the
        # fp32 error of a border take another code, one in thousands
        hq = dense.ffn_forward(xv, blk.wg, blk.wd, blk.layout, blk.act, blk.bg, blk.bd, rv if res is not None else None,
                               ALPHA, LIMIT, round_h=lambda h: dense.mxfp8_values(*dense.quantize_mxfp8(h)))["out"]
        rel = np.linalg.norm(got - hq) / np.linalg.norm(hq)
        say(f"  out against quantised h: {rel:.2e}")
        assert rel <= 2 * (RMS_BF if out_dtype == BF else 0.0) + 2e-3
    else:
        hb = dense.ffn_forward(xv, blk.wg, blk.wd, blk.layout, blk.act, blk.bg, blk.bd, rv if res is not None else None,
                               ALPHA, LIMIT, round_h=bf16_round_f64)["out"]
        # the same, with the 2-norm over everything: a rounding of h that falls the other way
        # happens to one value in hundreds, by a step of 2^-7
        rel = np.linalg.norm(got - hb) / np.linalg.norm(hb)
        say(f"  out against rounded h: {rel:.2e}")
        assert rel <= 2 * (RMS_BF if out_dtype == BF else 0.0) + 5e-4
    return got


@pytest.mark.parametrize("T,H,I,mx,clamped,bias", FFN_CASES)
def test_ffn_forward(T, H, I, mx, clamped, bias):
    blk = Block("fwd", H, I, mx, clamped, bias)
    ffn_check(blk, T, VARIANTS["auto"], BF, BF, True)
    fam = moe4.moe4_last_variant()
    assert fam in (moe4.MOE4_VARIANT_SKINNY, moe4.MOE4_VARIANT_TILED)
    for name in ("skinny", "tiled"):
        ffn_check(blk, T, VARIANTS[name], F32, F32 if T % 2 else None, False)
        assert moe4.moe4_last_variant() == VARIANTS[name]


@pytest.mark.parametrize("T,H,I,mx,clamped", [(4100, 72, 1544, False, False), (4099, 96, 1568, True, True),
                                              (2100, 1040, 2056, False, True), (1500, 2080, 1312, True, False)])
def test_ffn_forward_many_tiles(T, H, I, mx, clamped):
    # enough tiles for the largest tile shape, with ragged edges on every side
    blk = Block("big", H, I, mx, clamped, True)
    ffn_check(blk, T, VARIANTS["auto"], BF, BF, not mx)


@pytest.mark.parametrize("T,H,I,mx,clamped", [(70, 2056, 520, False, True), (130, 1032, 2072, False, False),
                                              (97, 2080, 1056, True, True), (200, 1056, 2080, True, False),
                                              (40, 4104, 136, False, True), (33, 8, 4104, False, False)])
def test_ffn_forward_split_k(T, H, I, mx, clamped):
    # few tiles and a long reduction: cut along k, ragged at the last part's end, and joined
    blk = Block("split", H, I, mx, clamped, True)
    ffn_check(blk, T, VARIANTS["tiled"], BF, BF, not mx)
    ffn_check(blk, T, VARIANTS["tiled"], F32, None, False)


@pytest.mark.parametrize("T,H,I", [(1, 96, 6176), (16, 64, 3104), (19, 32, 3136), (32, 96, 6144), (7, 6176, 32),
                                   (30, 6144, 96), (12, 12320, 32), (25, 12288, 64), (33, 64, 3104)])
def test_ffn_mx_few_tokens_wide(T, H, I):
    # every count of weight rows to a workgroup, in both products
    blk = Block("wide", H, I, True, T % 2 == 1, True)
    ffn_check(blk, T, VARIANTS["skinny"], BF, BF, True)
    ffn_check(blk, T, VARIANTS["skinny"], F32, None, False)


def test_ffn_mx_every_code_and_scale():
    # few tokens: each pre-activation is one code of one block times 1, which has to be exact
    H, I = 32, 1024
    codes = np.empty((2 * I, H), np.uint8)
    codes[:] = (32 * (np.arange(2 * I) // 256))[:, None] + np.arange(32)
    scales = (np.arange(2 * I) % 256).astype(np.uint8)[:, None]
    w = dense.mxfp8_values(codes, scales)   # NaN for code 0x7F, 0xFF and scale 255
    ffn = moe4.Ffn(moe4.MOE4_FFN_MXFP8, to_dev(codes), to_dev(np.zeros((H, I), np.uint8)), H=H, I=I,
                   gu_s=to_dev(scales), dn_s=to_dev(np.full((H, I // 32), 127, np.uint8)),
                   gu_layout=moe4.MOE4_GU_HALVES, act=moe4.MOE4_ACT_SWIGLU, variant=moe4.MOE4_VARIANT_SKINNY)
    x = np.zeros((H, H), np.uint8)
    x[np.arange(H), np.arange(H)] = 0x38   # 1.0
    gu = out_t((H, 2 * I), F32)
    out = torch.empty((H, H), dtype=F32, device="cuda")
    ws = torch.empty(moe4.moe4_ffn_workspace_size(ffn, H), dtype=torch.uint8, device="cuda")
    moe4.moe4_ffn_forward(ffn, to_dev(x), out, x_s=to_dev(np.full((H, 1), 127, np.uint8)), save_gu=gu.t, ws=ws)
    got, want = gu.t.double().cpu().numpy(), w.T
    bad = np.isnan(w).any(1)   # a NaN anywhere in a weight's row reaches every token
    assert bad.sum() == 256 * 2 + 6 and np.isnan(got[:, bad]).all()
    # a row with a value past fp32's range holds an infinity, which times 0 is a NaN: left out
    bad |= (np.abs(w) > 3.38e38).any(1)
    got, want = got[:, ~bad], want[:, ~bad]
    assert want.shape[1] >= 2048 - 518 - 8 * 8
    # below 2^-126 (fp32's and bf16's normal range) a value may be rounded or become zero
    small = np.abs(want) < 2.0 ** -126
    assert np.array_equal(got[~small], want[~small])
    assert np.all(np.abs(got[small] - want[small]) <= 2.0 ** -126)


def test_ffn_forward_in_place_residual():
    blk = Block("inplace", 264, 136)
    for T in (5, 200):
        x, _, _ = blk.tokens(T)
        res, _ = draw(rng("r", T), (T, 264))
        out = torch.empty_like(res)
        moe4.moe4_ffn_forward(blk.ffn, x, out, residual=res, ws=blk.ws(T))
        both = res.clone()
        moe4.moe4_ffn_forward(blk.ffn, x, both, residual=both, ws=blk.ws(T))
        assert torch.equal(out, both)


@pytest.mark.parametrize("variant", ["skinny", "tiled"])
@pytest.mark.parametrize("mx", [False, True])
def test_ffn_non_finite_tokens_stay_apart(mx, variant):
    # a NaN token, an infinite one, a NaN scale next to a row whose k ends inside a tile
    blk = Block("nan", 96, 64, mx, mx, True)
    T = 20
    x, xs, xv = blk.tokens(T)
    clean = torch.empty((T, 96), dtype=BF, device="cuda")
    moe4.moe4_ffn_forward(blk.ffn.with_variant(VARIANTS[variant]), x, clean, x_s=xs, ws=blk.ws(T))
    if mx:
        xs[7, 0] = 255
        x[11, 40] = 0x7F
    else:
        x[7, 3], x[11, 95] = float("nan"), float("inf")
    out = torch.empty_like(clean)
    moe4.moe4_ffn_forward(blk.ffn.with_variant(VARIANTS[variant]), x, out, x_s=xs, ws=blk.ws(T))
    o = val(out)
    keep = [t for t in range(T) if t not in (7, 11)]
    assert torch.equal(out[keep], clean[keep])
    assert np.isnan(o[7]).all() and not np.isfinite(o[11]).any()


BWD_CASES = [(1, 64, 32, False, False), (3, 72, 40, True, True), (16, 8, 8, False, True), (65, 264, 136, True, True),
             (127, 520, 264, False, False), (130, 136, 392, False, True), (300, 392, 200, True, False),
             (513, 264, 520, True, True), (1000, 72, 72, False, True)]


def ffn_backward_check(blk, T, wdt=BF, xdt=BF, add=True):
    x, _, xv = blk.tokens(T)
    r = rng("dy", T, blk.H)
    dy, dyv = draw(r, (T, blk.H), std=0.1)
    da, dav = draw(r, (T, blk.H), F32 if xdt == BF else BF, 0.1) if add else (None, 0.0)
    gv = dense.ffn_forward(xv, blk.wg, blk.wd, blk.layout, blk.act, blk.bg, blk.bd)["gu"].astype(np.float32)
    gu = to_dev(gv)
    H, I = blk.H, blk.I
    o = dict(dx=out_t((T, H), xdt), dw_gu=out_t((2 * I, H), wdt), dw_dn=out_t((H, I), wdt),
             db_gu=out_t((2 * I,), wdt), db_dn=out_t((H,), wdt))
    moe4.moe4_ffn_backward(blk.ffn, x, gu, dy, dx_add=da, ws=blk.ws(T, True), **{k: v.t for k, v in o.items()})
    w = dense.ffn_backward(xv, gv.astype(np.float64), dyv, blk.wg, blk.wd, blk.layout, blk.act, ALPHA, LIMIT)
    got = {k: val(v.t) for k, v in o.items()}
    for k, v in o.items():
        v.check(k)
        assert np.isfinite(got[k]).all(), k
    # 2-norms over each output: operands rounded to bf16 (one rounding; for db_dn none), the
    # output's own, and 1e-5 for the fp32 sums; small outputs spread more
    for k, rounds in (("dx", 1), ("dw_gu", 1), ("dw_dn", 1), ("db_gu", 1), ("db_dn", 0)):
        want = w[k] + (dav if k == "dx" else 0.0)
        dt = xdt if k == "dx" else wdt
        tol = 1.5 * (rounds * RMS_BF * np.linalg.norm(w[k]) +
                     (UBF if dt == BF else U32) * np.linalg.norm(want)) + 1e-5 * np.linalg.norm(w[k])
        if k in ("db_gu", "db_dn"):   # cancelling sums of T fp32 terms, and of T rounded ones
            terms = w["dgu"] if k == "db_gu" else dyv
            tol += np.linalg.norm((T * U32 + rounds * UBF) * np.abs(terms).sum(0))
        d = np.linalg.norm(got[k] - want)
        say(f"  {k}: {d:.3e} of {tol:.3e}")
        assert d <= tol, k
    # row by row, against the definition with the operands rounded as the kernel rounds them
    wr = dense.ffn_backward(xv, gv.astype(np.float64), dyv, blk.wg, blk.wd, blk.layout, blk.act, ALPHA, LIMIT,
                            exact=False)
    for k in ("dx", "dw_gu", "dw_dn"):
        want = wr[k] + (dav if k == "dx" else 0.0)
        dt = xdt if k == "dx" else wdt
        d = np.linalg.norm(got[k] - want, axis=1)
        tol = (ueps(dt) + 1e-5) * np.linalg.norm(want, axis=1) + 2e-3 * np.linalg.norm(wr[k], axis=1) + 1e-12
        assert np.all(d <= tol), (k, float(np.max(d / tol)))
    return got


@pytest.mark.parametrize("T,H,I,clamped,bias", BWD_CASES)
def test_ffn_backward(T, H, I, clamped, bias):
    blk = Block("bwd", H, I, False, clamped, bias)
    ffn_backward_check(blk, T)
    ffn_backward_check(blk, T, F32, F32, add=T % 2 == 0)


@pytest.mark.parametrize("T,H,I,clamped", [(4100, 1544, 264, True), (2050, 264, 2056, False), (9000, 520, 392, True),
                                         (4099, 136, 200, True), (2061, 392, 72, False)])
def test_ffn_backward_many_tiles(T, H, I, clamped):
    blk = Block("bwd-big", H, I, False, clamped, True)
    ffn_backward_check(blk, T)


def test_ffn_backward_outputs_one_by_one():
    # every subset of outputs gives the same bits as the call that wants all of them
    blk = Block("subset", 136, 72, False, True, True)
    T = 140
    x, _, xv = blk.tokens(T)
    dy, _ = draw(rng("dy1"), (T, 136), std=0.1)
    gu = to_dev(dense.ffn_forward(xv, blk.wg, blk.wd, blk.layout, blk.act, blk.bg, blk.bd)["gu"].astype(np.float32))
    shapes = dict(dx=(T, 136), dw_gu=(144, 136), dw_dn=(136, 72), db_gu=(144,), db_dn=(136,))

    def run(names):
        o = {k: torch.full(shapes[k], 7.0, dtype=BF, device="cuda") for k in names}
        moe4.moe4_ffn_backward(blk.ffn, x, gu, dy, ws=blk.ws(T, True), **o)
        return o
    full = run(shapes)
    for names in (["dx"], ["dw_gu"], ["dw_dn"], ["db_gu"], ["db_dn"], ["dx", "dw_dn"], ["dw_gu", "db_gu"]):
        for k, v in run(names).items():
            assert torch.equal(v, full[k]), (names, k)
    # dx on top of itself
    acc = full["dx"].clone()
    moe4.moe4_ffn_backward(blk.ffn, x, gu, dy, dx=acc, dx_add=acc, ws=blk.ws(T, True))
    want = val(full["dx"]) * 2
    assert np.linalg.norm(val(acc) - want) <= 3 * UBF * np.linalg.norm(want)


def test_ffn_backward_against_differences():
    # directional differences of the float64 forward; h and dGU are rounded once, out is fp32
    blk = Block("diff", 72, 48, False, True, True)
    T = 40
    x, _, xv = blk.tokens(T)
    dy, dyv = draw(rng("dyd"), (T, 72))
    fw = dense.ffn_forward(xv, blk.wg, blk.wd, blk.layout, blk.act, blk.bg, blk.bd)
    o = dict(dx=torch.empty((T, 72), device="cuda"), dw_gu=torch.empty((96, 72), device="cuda"),
             dw_dn=torch.empty((72, 48), device="cuda"))
    moe4.moe4_ffn_backward(blk.ffn, x, to_dev(fw["gu"].astype(np.float32)), dy, ws=blk.ws(T, True), **o)

    def loss(x=xv, wg=blk.wg, wd=blk.wd):
        return np.sum(dense.ffn_forward(x, wg, wd, blk.layout, blk.act, blk.bg, blk.bd)["out"] * dyv)
    r, h = rng("dir"), 1e-6
    for k, name, at in (("dx", "x", xv), ("dw_gu", "wg", blk.wg), ("dw_dn", "wd", blk.wd)):
        v = r.standard_normal(at.shape)
        want = (loss(**{name: at + h * v}) - loss(**{name: at - h * v})) / (2 * h)
        g = val(o[k])
        # independent relative errors of RMS_BF in the terms of a sum over random directions
        assert abs(np.sum(g * v) - want) <= 6 * RMS_BF * np.linalg.norm(g * v) + 1e-4 * abs(want), k


def test_ffn_no_tokens():
    blk = Block("empty", 72, 40, False, False, True)
    e = torch.empty((0, 72), dtype=BF, device="cuda")
    moe4.moe4_ffn_forward(blk.ffn, e, e)
    for dt in (BF, F32):
        o = dict(dw_gu=torch.full((80, 72), 3.0, dtype=dt, device="cuda"), dw_dn=torch.full((72, 40), 3.0, dtype=dt, device="cuda"),
                 db_gu=torch.full((80,), 3.0, dtype=dt, device="cuda"), db_dn=torch.full((72,), 3.0, dtype=dt, device="cuda"))
        moe4.moe4_ffn_backward(blk.ffn, e, torch.empty((0, 80), device="cuda"), e, dx=e, **o)
        assert all(bool((v == 0).all()) for v in o.values())
    moe4.moe4_add_rmsnorm(e, torch.ones(72, device="cuda"), 1e-6, out=e)
    dw = torch.full((72,), 3.0, device="cuda")
    moe4.moe4_add_rmsnorm_backward(e, e, torch.ones(72, device="cuda"), torch.empty(0, device="cuda"), e, dweight=dw)
    assert bool((dw == 0).all())


# ---------------------------------------------------------------- clipping

def grads_of(r, sizes, dtypes, std=1e-2):
    ts, vs = [], []
    for i, n in enumerate(sizes):
        t, v = draw(r, (n,), dtypes[i % len(dtypes)], std)
        ts.append(t), vs.append(v)
    return ts, vs


LISTS = [([5], [F32]), ([0, 1, 0, 3], [BF, F32]), ([8192, 8191, 8193, 16], [F32]), ([8192, 8191, 8193, 7], [BF]),
         ([100003] * 3, [F32, BF]), ([17] * 300, [F32, BF]), ([1 << 20] * 9, [F32]), ([0, 0], [F32])]


@pytest.mark.parametrize("sizes,dtypes", LISTS, ids=[f"{len(s)}x{max(s)}" for s, _ in LISTS])
@pytest.mark.parametrize("in_place", [False, True])
def test_clip_grads(sizes, dtypes, in_place):
    r = rng("clip", len(sizes), max(sizes))
    ts, vs = grads_of(r, sizes, dtypes)
    want = dense.grad_norm(vs)
    outs = None if in_place else [Guarded(tuple(t.shape), t.dtype) for t in ts]
    gl = moe4.GradList(ts, None if in_place else [o.t for o in outs])
    ws = torch.full((moe4.moe4_grad_workspace_size(gl),), 0xFF, dtype=torch.uint8, device="cuda")
    norm = torch.full((1,), -1.0, device="cuda")
    moe4.moe4_grad_norm(gl, norm, ws)
    # fp64 sums: the fp32 rounding of the root, and of the root's own step
    assert abs(norm.item() - want) <= 2 * U32 * want
    for max_norm in (max(want, 1.0) * 4, max(want, 1e-3) / 3):
        before = [t.clone() for t in ts]
        n2 = torch.full((1,), -1.0, device="cuda")
        moe4.moe4_clip_grads(gl, max_norm, n2, ws)
        cur = dense.grad_norm([val(t) for t in before])
        k = dense.clip_factor(cur, max_norm)
        assert abs(n2.item() - cur) <= 2 * U32 * cur
        for i, t in enumerate(before):
            got = ts[i] if in_place else outs[i].t
            if k == 1.0:
                assert torch.equal(got, t)
            else:   # the factor in fp32, its product, one rounding
                within(val(got), val(t) * k, (ueps(t.dtype) + 4 * U32) * np.abs(val(t)) * k + 1e-38, f"grad {i}")
            if not in_place:
                outs[i].check("clipped gradient")
                assert torch.equal(ts[i], t)
    # a norm from elsewhere
    total = torch.tensor([10.0 * max(want, 1.0)], device="cuda")
    before = [t.clone() for t in ts]
    n3 = torch.zeros(1, device="cuda")
    moe4.moe4_clip_grads(gl, 1.0, n3, norm_in=total)
    assert n3.item() == total.item()
    k = 1.0 / (total.item() + 1e-6)
    for i, t in enumerate(before):
        got = ts[i] if in_place else outs[i].t
        within(val(got), val(t) * k, (ueps(t.dtype) + 4 * U32) * np.abs(val(t)) * k + 1e-38, "given norm")


def test_grad_norm_of_extreme_values():
    # squares that overflow, or vanish, in fp32; infinities and NaNs leave the gradients alone
    for v in (1e30, 1e-30, 3e38):
        t = torch.full((1000,), v, device="cuda")
        gl = moe4.GradList([t])
        ws = torch.empty(moe4.moe4_grad_workspace_size(gl), dtype=torch.uint8, device="cuda")
        n = torch.empty(1, device="cuda")
        moe4.moe4_grad_norm(gl, n, ws)
        want = math.sqrt(1000) * float(np.float32(v))
        if want < 3.4028234e38:
            assert abs(n.item() - want) <= 2 * U32 * want
        else:
            assert math.isinf(n.item())
    for bad in (float("inf"), float("nan")):
        t = torch.ones(5000, device="cuda")
        t[4321] = bad
        o = torch.zeros_like(t)
        gl = moe4.GradList([t], [o])
        moe4.moe4_clip_grads(gl, 0.5, n, ws)
        assert not math.isfinite(n.item())
        assert torch.equal(o[:4321], t[:4321]) and torch.equal(o[4322:], t[4322:])


def test_sums_do_not_depend_on_the_run():
    # no atomics: the same bits from run to run
    blk = Block("det", 520, 264, False, True, True)
    T = 700
    x, _, xv = blk.tokens(T)
    dy, _ = draw(rng("dyx"), (T, 520))
    gu = to_dev(dense.ffn_forward(xv, blk.wg, blk.wd, blk.layout, blk.act, blk.bg, blk.bd)["gu"].astype(np.float32))
    w, _ = draw(rng("w"), (520,))
    rstd = torch.ones(T, device="cuda")
    nws = torch.empty(moe4.moe4_add_rmsnorm_workspace_size(T, 520), dtype=torch.uint8, device="cuda")
    first = None
    for _ in range(3):
        o = [torch.empty((528, 520), dtype=F32, device="cuda"), torch.empty((520, 264), dtype=F32, device="cuda"),
             torch.empty((528,), dtype=F32, device="cuda"), torch.empty((520,), dtype=F32, device="cuda")]
        moe4.moe4_ffn_backward(blk.ffn, x, gu, dy, dw_gu=o[0], dw_dn=o[1], db_gu=o[2], db_dn=o[3], ws=blk.ws(T, True))
        dx, dw = torch.empty((T, 520), dtype=BF, device="cuda"), torch.empty(520, device="cuda")
        moe4.moe4_add_rmsnorm_backward(dy, x, w, rstd, dx, dweight=dw, ws=nws)
        n = torch.empty(1, device="cuda")
        gl = moe4.GradList(o)
        moe4.moe4_grad_norm(gl, n, torch.empty(moe4.moe4_grad_workspace_size(gl), dtype=torch.uint8, device="cuda"))
        got = o + [dw, n]
        if first is None:
            first = got
        assert all(torch.equal(a, b) for a, b in zip(got, first))


# ----------------------------------------------------- refusals of the binding

def test_binding_refusals():
    x = torch.zeros((4, 64), dtype=BF, device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(ValueError, match="weight has shape"):
        moe4.moe4_add_rmsnorm(x, w[:32], 1e-6, out=x)
    with pytest.raises(TypeError, match="contiguous"):
        moe4.moe4_add_rmsnorm(x.t().contiguous().t(), w, 1e-6, out=x)
    with pytest.raises(TypeError, match="dtype"):
        moe4.moe4_add_rmsnorm(x.half(), w, 1e-6, out=x)
    with pytest.raises(TypeError, match="residual's dtype"):
        moe4.moe4_add_rmsnorm(x, w, 1e-6, residual=x, sum_out=x.float(), out=x)
    with pytest.raises(ValueError, match="out_s has shape"):
        moe4.moe4_add_rmsnorm(x, w, 1e-6, out_q=x.to(torch.uint8), out_s=torch.zeros((4, 3), dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError, match="GPU"):
        moe4.moe4_add_rmsnorm(x, w.cpu(), 1e-6, out=x)
    blk = Block("refuse", 64, 32)
    with pytest.raises(moe4.Moe4Error, match="workspace"):
        moe4.moe4_ffn_forward(blk.ffn, x, x.clone())
    with pytest.raises(ValueError, match="x has shape"):
        moe4.moe4_ffn_forward(blk.ffn, x[:, :32].contiguous(), x.clone(), ws=blk.ws(4))
    with pytest.raises(TypeError, match="one dtype"):
        moe4.moe4_ffn_backward(blk.ffn, x, torch.zeros((4, 64), device="cuda"), x, dw_gu=torch.empty((64, 64), dtype=BF, device="cuda"),
                               dw_dn=torch.empty((64, 32), device="cuda"), ws=blk.ws(4, True))
    with pytest.raises(ValueError, match="w_dn has shape"):
        moe4.Ffn(moe4.MOE4_FFN_BF16, torch.empty((64, 64), dtype=BF, device="cuda"), torch.empty((64, 64), dtype=BF, device="cuda"),
                 gu_layout=1, act=1, H=64, I=32)
    with pytest.raises(moe4.Moe4Error, match="16-byte"):
        moe4.moe4_quantize_mxfp8(torch.zeros(40, dtype=BF, device="cuda")[4:36], torch.empty(32, dtype=torch.uint8, device="cuda"),
                                 torch.empty(1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError, match="outs\\[0\\] has dtype"):
        moe4.GradList([x], [w])
    with pytest.raises(ValueError, match="outs\\[0\\] has shape"):
        moe4.GradList([x], [x[:2]])


# ------------------------------------------------------------ as they are used

def test_graph_capture_of_the_dense_step():
    # norm, block, norm; backward; clipping: captured once, replayed on new inputs, with eager
    # work between the replays
    blk = Block("graph", 264, 136, False, True, True)
    T, H, I = 130, 264, 136
    w, _ = draw(rng("gw"), (H,))
    z = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype, device="cuda")   # noqa: E731
    b = dict(x=z(T, H), res=z(T, H), dy=z(T, H), s=z(T, H), n=z(T, H), r=z(T, dtype=F32), gu=z(T, 2 * I, dtype=F32), o=z(T, H),
             dn=z(T, H), dx=z(T, H), dw=z(H, dtype=F32), wg=z(2 * I, H), wd=z(H, I), bg=z(2 * I), bd=z(H), norm=z(1, dtype=F32))
    gl = moe4.GradList([b["wg"], b["wd"], b["bg"], b["bd"], b["dw"]])
    ws = blk.ws(T, True)
    nws = torch.empty(moe4.moe4_add_rmsnorm_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    gws = torch.empty(moe4.moe4_grad_workspace_size(gl), dtype=torch.uint8, device="cuda")

    def step():
        moe4.moe4_add_rmsnorm(b["x"], w, 1e-6, residual=b["res"], sum_out=b["s"], out=b["n"], rstd=b["r"])
        moe4.moe4_ffn_forward(blk.ffn, b["n"], b["o"], residual=b["s"], save_gu=b["gu"], ws=ws)
        moe4.moe4_ffn_backward(blk.ffn, b["n"], b["gu"], b["dy"], dx=b["dn"], dw_gu=b["wg"], dw_dn=b["wd"], db_gu=b["bg"],
                               db_dn=b["bd"], ws=ws)
        moe4.moe4_add_rmsnorm_backward(b["dn"], b["s"], w, b["r"], b["dx"], dres=b["dy"], dweight=b["dw"], ws=nws)
        moe4.moe4_clip_grads(gl, 0.5, b["norm"], gws)

    def fill(k):
        r = rng("fill", k)
        for name in ("x", "res", "dy"):
            b[name].copy_(draw(r, (T, H))[0])
    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    keys = [k for k in b if k not in ("x", "res", "dy")]
    for k in range(1, 5):
        fill(k)
        g.replay()
        torch.cuda.synchronize()
        got = {n: b[n].clone() for n in keys}
        for n in keys:
            b[n].fill_(float("nan"))
        step()     # eager, between replays
        torch.cuda.synchronize()
        for n in keys:
            assert torch.equal(got[n], b[n]), (k, n)


@pytest.mark.parametrize("T,H,I,mx", [(2600, 264, 2568, False), (2600, 288, 2592, True), (200, 2080, 544, True),
                                      (20, 288, 160, True)])
def test_graph_capture_of_every_kernel_family(T, H, I, mx):
    # large tiles, split products, skinny kernels: captured without an eager call before
    blk = Block("capture", H, I, mx, mx, True)
    x, xs, _ = blk.tokens(T)
    out, base = torch.zeros((T, H), dtype=BF, device="cuda"), torch.zeros((T, H), dtype=BF, device="cuda")
    ws = blk.ws(T)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe4.moe4_ffn_forward(blk.ffn, x, out, x_s=xs, ws=ws)
    for k in range(3):
        x2, xs2, _ = blk.tokens(T, k + 1)
        x.copy_(x2)
        if mx:
            xs.copy_(xs2)
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        moe4.moe4_ffn_forward(blk.ffn, x, base, x_s=xs, ws=ws)
        assert torch.equal(got, base)


def test_offsets_past_32_bits():
    # tensors of more than 2^32 bytes: the last rows are those of a call on them alone
    H, T, tail = 2048, 1_060_000, 300
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((T, H), generator=gen, device="cuda", dtype=BF)
    w = torch.ones(H, device="cuda")
    out = torch.empty_like(x)
    q, s = torch.empty((T, H), dtype=torch.uint8, device="cuda"), torch.empty((T, H // 32), dtype=torch.uint8, device="cuda")
    rstd = torch.empty(T, device="cuda")
    moe4.moe4_add_rmsnorm(x, w, 1e-6, out=out, out_q=q, out_s=s, rstd=rstd)
    xe = x[-tail:].clone()
    o2, r2 = torch.empty_like(xe), torch.empty(tail, device="cuda")
    q2, s2 = torch.empty((tail, H), dtype=torch.uint8, device="cuda"), torch.empty((tail, H // 32), dtype=torch.uint8, device="cuda")
    moe4.moe4_add_rmsnorm(xe, w, 1e-6, out=o2, out_q=q2, out_s=s2, rstd=r2)
    # (another number of rows takes another split of the row's sum: bf16 steps apart at most)
    assert torch.allclose(rstd[-tail:], r2, rtol=1e-5, atol=0)
    assert torch.allclose(out[-tail:].float(), o2.float(), rtol=2.0 ** -7, atol=0)
    moe4.moe4_quantize_mxfp8(x, q, s)
    moe4.moe4_quantize_mxfp8(xe, q2, s2)
    assert torch.equal(q[-tail:], q2) and torch.equal(s[-tail:], s2)
    dx = torch.empty_like(x)
    moe4.moe4_add_rmsnorm_backward(out, x, w, rstd, dx)
    d2 = torch.empty_like(xe)
    moe4.moe4_add_rmsnorm_backward(out[-tail:].clone(), xe, w, rstd[-tail:].clone(), d2)
    # dy is the normalised row itself, so p and n mean(p n) all but cancel and what is left is no
    # measure: as in the parity test, each call's fp32 error is at most e times the terms'
    # magnitudes rstd (|p| + |n| mean|p n|), and a bf16 step lies between their roundings
    p, n, rr = out[-tail:].double(), xe.double() * r2.double()[:, None], r2.double()[:, None]
    mag = rr * (p.abs() + n.abs() * (p * n).abs().mean(1, keepdim=True))
    tol = 2 * (512 + 24) * U32 * mag + 2.0 ** -7 * d2.double().abs()
    assert bool(((dx[-tail:].double() - d2.double()).abs() <= tol).all())
    del dx, q, s
    blk = Block("huge", H, 16)
    moe4.moe4_ffn_forward(blk.ffn, x, out, ws=blk.ws(T))
    o2 = torch.empty_like(xe)
    moe4.moe4_ffn_forward(blk.ffn.with_variant(VARIANTS["tiled"]), xe, o2, ws=blk.ws(tail))
    # (few tokens are split along k: the fp32 sums' order, then one bf16 step of h and out)
    d = (out[-tail:].float() - o2.float()).norm()
    assert d <= 4 * RMS_BF * o2.float().norm()


def test_other_streams():
    # a side stream, by argument and as the current one, ordered by events alone
    blk = Block("stream", 136, 72)
    T = 100
    x, _, _ = blk.tokens(T)
    base = torch.empty((T, 136), dtype=BF, device="cuda")
    moe4.moe4_ffn_forward(blk.ffn, x, base, ws=blk.ws(T))
    st = torch.cuda.Stream()
    a, c = torch.empty_like(base), torch.empty_like(base)
    wa, wc = blk.ws(T), blk.ws(T)
    st.wait_stream(torch.cuda.current_stream())
    moe4.moe4_ffn_forward(blk.ffn, x, a, ws=wa, stream=st)
    with torch.cuda.stream(st):
        moe4.moe4_ffn_forward(blk.ffn, x, c, ws=wc)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(a, base) and torch.equal(c, base)


def test_block_with_routed_experts():
    """The whole block as it is used: residual norm, router, routed 4-bit experts and combine,
    the dense block with the stream in its epilogue, the next layer's norm taking the routed
    output; then back through the dense block and the norm."""
    import oracle
    from bit_mixture_experts_amd import inputs as inp
    from gpu_helpers import run_layer
    from test_gpu_parity import QWEN_SMALL, layer_of
    spec = QWEN_SMALL
    L = layer_of(spec)
    ex = L.device()
    T, H, I, k = 37, spec.H, 192, spec.k
    blk = Block("shared", H, I)
    r = rng("whole")
    x, xv = draw(r, (T, H))
    res, rv = draw(r, (T, H))
    w1, w1v = draw(r, (H,))
    w2, w2v = draw(r, (H,))
    wr, wrv = draw(r, (spec.E, H), std=1 / math.sqrt(H))
    h = torch.empty((T, H), dtype=BF, device="cuda")
    n = torch.empty_like(h)
    rstd = torch.empty(T, device="cuda")
    moe4.moe4_add_rmsnorm(x, w1, 1e-6, residual=res, sum_out=h, out=n, rstd=rstd)
    lg = torch.empty((T, spec.E), device="cuda")
    moe4.moe4_router_logits(n, wr, lg)
    routed = run_layer(ex, n, lg, k)
    gu = torch.empty((T, 2 * I), device="cuda")
    stream = torch.empty_like(h)
    moe4.moe4_ffn_forward(blk.ffn, n, stream, residual=h, save_gu=gu, ws=blk.ws(T))
    h2, n2 = torch.empty_like(h), torch.empty_like(h)
    moe4.moe4_add_rmsnorm(routed["out32"], w2, 1e-6, residual=stream, sum_out=h2, out=n2)
    # the float64 block on the bf16 values the GPU's own steps pass on
    sv, rs, yv = dense.add_rmsnorm(xv, w1v, 1e-6, rv, bf16_round_f64)
    assert np.array_equal(sv, val(h))
    nv = val(n)
    within(nv, yv, (UBF + 2 * norm_bound(H)) * np.abs(yv) + 1e-38, "first norm")
    ri, rw = oracle.route(lg.cpu().numpy(), k)
    ro = oracle.layer_forward(bits(n), ri, rw, L.W)["out"]
    fo = dense.ffn_forward(nv, blk.wg, blk.wd, blk.layout, blk.act, residual=sv)
    want = fo["out"] + ro
    s2 = val(h2)
    row_norm(s2, want, 2e-2, "stream after the block")
    _, _, y2 = dense.add_rmsnorm(s2, w2v, 1e-6)
    within(val(n2), y2, (UBF + 2 * norm_bound(H)) * np.abs(y2) + 1e-38, "second norm")
    # backward: the stream's gradient through the dense block (a routed part added), the norm
    dy, dyv = draw(r, (T, H), std=0.1)
    droute, drv = draw(r, (T, H), F32, 0.1)
    dn = torch.empty((T, H), device="cuda")
    dwg, dwd = torch.empty((2 * I, H), device="cuda"), torch.empty((H, I), device="cuda")
    moe4.moe4_ffn_backward(blk.ffn, n, gu, dy, dx=dn, dx_add=droute, dw_gu=dwg, dw_dn=dwd, ws=blk.ws(T, True))
    dx, dw = torch.empty_like(h), torch.empty(H, device="cuda")
    nws = torch.empty(moe4.moe4_add_rmsnorm_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    moe4.moe4_add_rmsnorm_backward(dn, h, w1, rstd, dx, dres=dy, dweight=dw, ws=nws)
    b = dense.ffn_backward(nv, fo["gu"], dyv, blk.wg, blk.wd, blk.layout, blk.act)
    wx, ww = dense.add_rmsnorm_backward(b["dx"] + drv, sv, w1v, rs, dyv)
    row_norm(val(dx), wx, 2 * (UBF + RMS_BF), "gradient of the stream")
    assert np.linalg.norm(dw.double().cpu().numpy() - ww) <= 2 * RMS_BF * np.linalg.norm(ww) + 1e-5
    grads = [dwg, dwd, dw]
    gl = moe4.GradList(grads)
    total = dense.grad_norm([val(g) for g in grads])
    norm = torch.empty(1, device="cuda")
    moe4.moe4_clip_grads(gl, total / 2, norm, torch.empty(moe4.moe4_grad_workspace_size(gl), dtype=torch.uint8, device="cuda"))
    assert abs(norm.item() - total) <= 2 * U32 * total
    assert abs(dense.grad_norm([val(g) for g in grads]) - total / 2) <= 1e-5 * total


def test_clip_refuses_outputs_that_overlap():
    a = torch.arange(64, dtype=F32, device="cuda")
    norm, ws = torch.empty(1, dtype=F32, device="cuda"), None
    before = a.clone()
    twice = moe4.GradList([a, torch.ones(4, device="cuda"), a])
    ws = torch.empty(moe4.moe4_grad_workspace_size(twice), dtype=torch.uint8, device="cuda")
    # read only, a gradient counts as often as it is in the list: sum i^2 for i < 64 is 85344
    moe4.moe4_grad_norm(twice, norm, ws)
    assert abs(norm.item() - (2 * 85344 + 4) ** 0.5) <= 2.0 ** -23 * norm.item()
    b = torch.empty(64, dtype=F32, device="cuda")
    refused = [(twice, "outs\\[2\\] overlaps entry 0"),
               (moe4.GradList([a[:32], a[16:48]]), "outs\\[1\\] overlaps entry 0"),
               (moe4.GradList([a, b], [b, a]), "overlaps entry"),
               (moe4.GradList([a[:32], a[32:]], [b[:32], b[16:48]]), "outs\\[1\\] overlaps entry 0"),
               (moe4.GradList([a[16:48]], [a[:32]]), "overlaps entry 0")]
    for g, what in refused:
        with pytest.raises(ValueError, match=what):
            moe4.moe4_clip_grads(g, 1.0, norm, ws)
    torch.cuda.synchronize()
    assert torch.equal(a, before)
    # neighbours, a gradient read by two entries, and in place beside out of place
    ok = moe4.GradList([a[:32], a[32:], a[:32]], [a[:32], b[:32], b[32:]])
    assert ok.clash is not None   # entry 2 reads what entry 0 writes
    ok = moe4.GradList([a[:32], a[32:], a[32:]], [a[:32], b[:32], b[32:]])
    moe4.moe4_clip_grads(ok, 1e9, norm, ws)
    assert torch.equal(b[:32], a[32:]) and torch.equal(b[32:], a[32:]) and torch.equal(a, before)
    moe4.moe4_clip_grads(moe4.GradList([a[:32], a[32:]]), 1e9, norm, ws)


def test_quantize_refuses_a_scalar():
    x = torch.ones((), dtype=F32, device="cuda")
    with pytest.raises(ValueError, match="no dimension"):
        moe4.moe4_quantize_mxfp8(x, x, x)
