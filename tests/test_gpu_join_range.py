"""The join's norm of the block's output at the ends of fp32's range: b * rstd is taken first, as the
definition says, so that neither b * w_post nor a rstd of 0 leaves it."""
import numpy as np
import pytest
import torch

from gpu_helpers import to_dev
from oracle import block4
from test_gpu_dense import BF, F32, U32, draw, moe4, rng, val, within

pytestmark = pytest.mark.gpu

# (rows, columns): one to sixteen waves a row
SHAPES = [(3, 64), (2049, 512), (2049, 2880), (5, 2880), (2, 16384)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,H", SHAPES)
def test_rows_past_the_sum_of_squares_give_rstd_0(T, H, dtype):
    # (b * w_post would be an infinity, and 0 times it a NaN)
    r = rng("range", T, H)
    b, _ = draw(r, (T, H), dtype)
    res, rv = draw(r, (T, H))
    b[1, ::3], b[1, 1::3], b[1, 2::3] = 3e38, -3e38, 1.0
    w = torch.full((H,), 2.0, dtype=dtype, device="cuda")
    s, ro = torch.empty((T, H), dtype=BF, device="cuda"), torch.empty(T, device="cuda")
    moe4.moe4_join_norm(b, None, 1e-6, residual=res, w_post=w, sum_out=s, rstd_post=ro)
    assert float(ro[1]) == 0.0 and torch.equal(s[1], res[1])
    assert bool(s.isfinite().all())


@pytest.mark.parametrize("T,H", SHAPES)
def test_large_rows_and_weights(T, H):
    # squares inside fp32's range, b * w_post far outside
    r = rng("large", T, H)
    bv = (r.choice([-1.0, 1.0], (T, H)) * r.uniform(1, 2, (T, H)) * 1e16).astype(np.float32)
    wv = (r.uniform(1, 2, H) * 1e25).astype(np.float32)
    b, w = to_dev(bv), to_dev(wv)
    s = torch.empty((T, H), device="cuda")
    moe4.moe4_join_norm(b, None, 1e-6, w_post=w, block_scale=0.5, sum_out=s)
    want = block4.join_norm(bv.astype(np.float64), block_scale=0.5, w_post=wv.astype(np.float64), eps=1e-6)["s"]
    # the sum of H squares (half a step an addition, halved by the root), root, factors, products
    within(val(s), want, ((H + 8) * U32 / 2 + 8 * U32) * np.abs(want), "s")
