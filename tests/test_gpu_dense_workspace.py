"""One workspace, made for the largest batch, serves every smaller one: same results as with a
workspace of the call's own, and nothing written behind the bytes asked for."""
import numpy as np
import pytest
import torch

from oracle import dense
from test_gpu_dense import BF, F32, Block, draw, rng

pytestmark = pytest.mark.gpu
moe4 = pytest.importorskip("bit_mixture_experts_amd.moe4")


class Scratch:
    """n bytes full of NaNs with a band of sentinels behind them."""

    def __init__(self, n):
        self.raw = torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
        self.raw[n:] = 0xA5
        self.ws = self.raw[:n]

    def check(self):
        assert bool((self.raw[self.ws.numel():] == 0xA5).all())


# sizes at which products are cut along k for few tokens, and whole for many
@pytest.mark.parametrize("H,I,mx", [(2056, 136, False), (1032, 2056, False), (136, 2056, False), (2080, 160, True),
                                    (1056, 2080, True)])
def test_block_with_the_largest_batchs_workspace(H, I, mx):
    blk = Block("ws", H, I, mx, False, True)
    tokens = (4200, 2100, 1025, 513, 128, 70, 1)
    sizes = {(T, b): moe4.moe4_ffn_workspace_size(blk.ffn, T, b) for T in tokens for b in (False, True)}
    shared = {b: Scratch(max(sizes[T, b] for T in tokens[:1])) for b in (False, True)}
    for T in tokens:
        x, xs, xv = blk.tokens(T)
        outs = []
        for sc in (shared[False], Scratch(sizes[T, False])):
            out = torch.full((T, H), float("nan"), dtype=F32, device="cuda")
            moe4.moe4_ffn_forward(blk.ffn.with_variant(moe4.MOE4_VARIANT_TILED), x, out, x_s=xs, ws=sc.ws)
            sc.check()
            outs.append(out)
        assert torch.equal(*outs), T
        if mx:
            continue
        dy, _ = draw(rng("ws-dy", T, H), (T, H), std=0.1)
        gu = torch.from_numpy(dense.ffn_forward(xv, blk.wg, blk.wd, blk.layout, blk.act, blk.bg)["gu"].astype(np.float32)).cuda()
        grads = []
        for sc in (shared[True], Scratch(sizes[T, True])):
            o = dict(dx=torch.empty((T, H), dtype=BF, device="cuda"), dw_gu=torch.empty((2 * I, H), dtype=F32, device="cuda"),
                     dw_dn=torch.empty((H, I), dtype=F32, device="cuda"), db_gu=torch.empty((2 * I,), dtype=F32, device="cuda"),
                     db_dn=torch.empty((H,), dtype=F32, device="cuda"))
            moe4.moe4_ffn_backward(blk.ffn, x, gu, dy, ws=sc.ws, **o)
            sc.check()
            grads.append(o)
        for k in grads[0]:
            assert torch.equal(grads[0][k], grads[1][k]), (T, k)
            assert bool(torch.isfinite(grads[0][k]).all()), (T, k)


@pytest.mark.parametrize("H", [520, 2048, 2056])
def test_norm_backward_with_the_largest_batchs_workspace(H):
    big = 4100
    shared = Scratch(moe4.moe4_add_rmsnorm_workspace_size(big, H))
    r = rng("ws-norm", H)
    dy, _ = draw(r, (big, H), std=0.1)
    s, sv = draw(r, (big, H))
    w, _ = draw(r, (H,))
    rstd = torch.from_numpy((1 / np.sqrt(np.mean(sv * sv, 1))).astype(np.float32)).cuda()
    for T in (big, 2048, 2047, 1025, 3, 1):
        outs = []
        for sc in (shared, Scratch(moe4.moe4_add_rmsnorm_workspace_size(T, H))):
            dx, dw = torch.empty((T, H), dtype=BF, device="cuda"), torch.full((H,), float("nan"), device="cuda")
            moe4.moe4_add_rmsnorm_backward(dy[:T], s[:T], w, rstd[:T], dx, dweight=dw, ws=sc.ws)
            sc.check()
            outs.append((dx, dw))
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
        assert bool(torch.isfinite(outs[0][1]).all())
