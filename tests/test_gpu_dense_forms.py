"""The dense feed-forward block in every pairing of gate/up layout and activation, and the
precision of its MXFP8 products for few tokens, against the float64 definitions in
oracle/dense.py."""
import numpy as np
import pytest
import torch

from oracle import dense
from gpu_helpers import to_dev
from test_gpu_dense import BF, F32, U32, VARIANTS, Block, ffn_backward_check, ffn_check, out_t, rng, within

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


# ----------------------------------------------------------------- backward

# dH whole in small tiles; cut along k and joined; dH and the other products in the largest tiles
BWD = [(65, 264, 136), (300, 392, 200), (1, 1544, 72), (70, 1032, 136), (333, 2056, 40), (1030, 1024, 264)]


@pytest.mark.parametrize("layout,act", FORMS)
@pytest.mark.parametrize("T,H,I", BWD + [(4100, 1032, 2056)])
def test_ffn_backward_forms(T, H, I, layout, act):
    ffn_backward_check(Form("form-bwd", H, I, layout, act, bias=True), T)
