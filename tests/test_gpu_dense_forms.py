"""The dense feed-forward block in every pairing of gate/up layout and activation, and the
precision of its bias gradient and of the MXFP8 products for few tokens, against the float64
definitions in oracle/dense.py."""
import math

import numpy as np
import pytest
import torch

from oracle import bf16_bits_from_f32, bf16_bits_to_f64, dense
from gpu_helpers import say, to_dev
from test_gpu_dense import (ALPHA, BF, F32, LIMIT, U32, UBF, VARIANTS, Block, draw, ffn_backward_check, ffn_check,
                            out_t, rng, val, within)

pytestmark = pytest.mark.gpu
moe4 = pytest.importorskip("bit_mixture_experts_amd.moe4")

LAYOUTS = {"halves": moe4.MOE4_GU_HALVES, "interleaved": moe4.MOE4_GU_INTERLEAVED}
FORMS = [(layout, act) for layout in ("halves", "interleaved") for act in ("swiglu", "clamped")]


class Form(Block):
    """A block whose layout does not follow from its activation."""

    def __init__(self, key, H, I, layout, act, mx=False, bias=False):
        super().__init__(key, H, I, mx, act == "clamped", bias)
        self.layout = layout
        self.ffn.desc.gu_layout = LAYOUTS[layout]


# ------------------------------------------------------------------ forward

@pytest.mark.parametrize("layout,act", FORMS)
@pytest.mark.parametrize("T,H,I,mx", [(1, 72, 40, False), (19, 264, 136, False), (50, 136, 520, False),
                                      (3, 96, 96, True), (27, 224, 160, True), (70, 160, 288, True)])
def test_ffn_forward_forms(T, H, I, mx, layout, act):
    blk = Form("form", H, I, layout, act, mx, True)
    for name in ("skinny", "tiled"):
        ffn_check(blk, T, VARIANTS[name], BF, BF, True)
        assert moe4.moe4_last_variant() == VARIANTS[name]


@pytest.mark.parametrize("layout,act", FORMS)
@pytest.mark.parametrize("T,H,I,mx", [(70, 2056, 136, False), (97, 2080, 160, True),      # cut along k
                                      (2100, 136, 2056, False), (2100, 160, 2080, True)])   # the largest tiles
def test_ffn_forward_forms_split_and_large(T, H, I, mx, layout, act):
    ffn_check(Form("form-big", H, I, layout, act, mx, True), T, VARIANTS["tiled"], BF, BF, True)


def test_ffn_mx_few_tokens_multiply_exactly():
    """Products of e4m3 values whose sizes are 2^17 apart within a block of 32: an instruction that
    keeps each only to 2^-16 of the largest loses the small ones, fp32 sums do not. The bound is
    fp32's: one rounding of every partial sum."""
    H, I, T = 64, 32, 16
    r = rng("mx-exact")
    x = np.full((T, H), 0x01, np.uint8)                          # 2^-9
    x[np.arange(T), r.integers(0, 32, T)] = 0x78                 # 256
    x[np.arange(T), 32 + r.integers(0, 32, T)] = 0xF8            # -256 in the other block
    w = (0x38 + r.integers(0, 8, (2 * I, H))).astype(np.uint8)   # 1 .. 1.875
    one = lambda *s: to_dev(np.full(s, 127, np.uint8))           # noqa: E731
    ffn = moe4.Ffn(moe4.MOE4_FFN_MXFP8, to_dev(w), to_dev(np.zeros((H, I), np.uint8)), H=H, I=I, gu_s=one(2 * I, H // 32),
                   dn_s=one(H, I // 32), gu_layout=moe4.MOE4_GU_HALVES, act=moe4.MOE4_ACT_SWIGLU,
                   variant=moe4.MOE4_VARIANT_SKINNY)
    gu, out = out_t((T, 2 * I), F32), torch.empty((T, H), dtype=F32, device="cuda")
    ws = torch.empty(moe4.moe4_ffn_workspace_size(ffn, T), dtype=torch.uint8, device="cuda")
    moe4.moe4_ffn_forward(ffn, to_dev(x), out, x_s=one(T, H // 32), save_gu=gu.t, ws=ws)
    s = np.full((1, H // 32), 127, np.uint8)
    xv, wv = dense.mxfp8_values(x, s.repeat(T, 0)), dense.mxfp8_values(w, s.repeat(2 * I, 0))
    # the small products together are far above the bound: losing them shows
    small = np.abs(xv) < 1
    assert ((xv * small) @ wv.T).min() > 4 * ((H + 2) * U32 * (np.abs(xv) @ wv.T)).max()
    within(gu.t.double().cpu().numpy(), xv @ wv.T, (H + 2) * U32 * (np.abs(xv) @ np.abs(wv).T), "gu")


@pytest.mark.parametrize("mx", [False, True])
def test_ffn_small_block_many_tokens_runs_tiled(mx):
    # a small block's weights are read again for every few tokens: with many tokens the tiles win
    blk = Form("small", 64, 64, "halves", "swiglu", mx, True)
    for T, family in ((64, moe4.MOE4_VARIANT_SKINNY), (16384, moe4.MOE4_VARIANT_TILED)):
        ffn_check(blk, T, VARIANTS["auto"], BF, BF, True)
        assert moe4.moe4_last_variant() == family


# ----------------------------------------------------------------- backward

# dH whole in small tiles; cut along k and joined; dH and the other products in the largest tiles
BWD = [(65, 264, 136), (300, 392, 200), (1, 1544, 72), (70, 1032, 136), (333, 2056, 40), (1030, 1024, 264)]


@pytest.mark.parametrize("layout,act", FORMS)
@pytest.mark.parametrize("T,H,I", BWD + [(4100, 1032, 2056)])
def test_ffn_backward_forms(T, H, I, layout, act):
    ffn_backward_check(Form("form-bwd", H, I, layout, act, bias=True), T)


def grad_terms(gv, dh, layout, act):
    """(dGU, the size of its terms, what the activation's evaluation in fp32 may cost in units
    of 2^-24 of that): each [T, 2I] in memory's order."""
    g, u = dense._split(gv, layout)
    if act == "swiglu":
        a, lin, sat_g, sat_u = 1.0, u, np.zeros(g.shape, bool), np.zeros(g.shape, bool)
    else:
        a, lin = ALPHA, np.clip(u, -LIMIT, LIMIT) + 1
        sat_g, sat_u = g > LIMIT, np.abs(u) > LIMIT
        g = np.where(sat_g, LIMIT, g)
    s = 1 / (1 + np.exp(-a * g))
    dg, du = np.where(sat_g, 0.0, dh * lin * (s + a * g * s * (1 - s))), np.where(sat_u, 0.0, dh * g * s)
    mg = np.where(sat_g, 0.0, np.abs(dh) * np.abs(lin) * (s + np.abs(a * g) * s * (1 - s)))
    # the exponential's argument is off by three roundings of |a g|, which is its relative error;
    # about eight more operations, and 1 - s, off by 3 * 2^-24 of s times |a g|
    cost = 16 + 8 * np.abs(a * g)
    return (dense._join(dg, du, layout), dense._join(mg, np.abs(du), layout), dense._join(cost, cost, layout))


@pytest.mark.parametrize("layout,act", FORMS)
@pytest.mark.parametrize("T,H,I", BWD)
def test_ffn_bias_gradient_is_summed_in_fp32(T, H, I, layout, act):
    """db_gu sums dGU before its rounding to bf16, whatever the number of tokens. One entry of dY
    a token, so that dH is one exact product; then only the activation's own fp32 operations
    and the T fp32 additions are left."""
    blk = Form("form-db", H, I, layout, act, bias=True)
    r = rng("onehot", T, H)
    dyv = np.zeros((T, H))
    dyv[np.arange(T), r.integers(0, H, T)] = bf16_bits_to_f64(bf16_bits_from_f32(r.standard_normal(T).astype(np.float32)))
    x, _, xv = blk.tokens(T)
    gv = dense.ffn_forward(xv, blk.wg, blk.wd, blk.layout, blk.act, blk.bg, blk.bd)["gu"].astype(np.float32)
    dy = to_dev(bf16_bits_from_f32(dyv.astype(np.float32)))
    alone, full = out_t((2 * I,), F32), out_t((2 * I,), F32)
    moe4.moe4_ffn_backward(blk.ffn, x, to_dev(gv), dy, db_gu=alone.t, ws=blk.ws(T, True))
    dx, dwg = torch.empty((T, H), dtype=BF, device="cuda"), torch.empty((2 * I, H), dtype=F32, device="cuda")
    dwd = torch.empty((H, I), dtype=F32, device="cuda")
    moe4.moe4_ffn_backward(blk.ffn, x, to_dev(gv), dy, dx=dx, dw_gu=dwg, dw_dn=dwd, db_gu=full.t, ws=blk.ws(T, True))
    alone.check("db_gu"), full.check("db_gu")
    assert torch.equal(alone.t, full.t)
    dgu, mag, cost = grad_terms(gv.astype(np.float64), dyv @ blk.wd, layout, act)
    tol = U32 * ((cost + T + 4) * mag).sum(0) + 1e-37
    within(full.t.double().cpu().numpy(), dgu.sum(0), tol, "db_gu")


@pytest.mark.parametrize("layout,act", FORMS)
@pytest.mark.parametrize("T,H,I", BWD[:4])
def test_ffn_bias_gradient_of_ordinary_gradients(T, H, I, layout, act):
    # the 2-norm over the output: 1e-5 for the fp32 sums of dH, T more fp32 additions
    blk = Form("form-db2", H, I, layout, act, bias=True)
    x, _, xv = blk.tokens(T)
    dy, dyv = draw(rng("dy-db", T, H), (T, H), std=0.1)
    gv = dense.ffn_forward(xv, blk.wg, blk.wd, blk.layout, blk.act, blk.bg, blk.bd)["gu"].astype(np.float32)
    w = dense.ffn_backward(xv, gv.astype(np.float64), dyv, blk.wg, blk.wd, layout, act, ALPHA, LIMIT)
    for dt in (F32, BF):
        db = out_t((2 * I,), dt)
        moe4.moe4_ffn_backward(blk.ffn, x, to_dev(gv), dy, db_gu=db.t, ws=blk.ws(T, True))
        db.check("db_gu")
        d = np.linalg.norm(val(db.t) - w["db_gu"])
        tol = ((UBF if dt == BF else U32) + 1e-5) * np.linalg.norm(w["db_gu"]) + \
            np.linalg.norm(T * U32 * np.abs(w["dgu"]).sum(0))
        say(f"  db_gu: {d:.3e} of {tol:.3e}")
        assert d <= tol and math.isfinite(d)
