"""The ends of the range in which the operands of the dense MXFP4 product are exact, as moe4.h states
them: one weight times one activation, both powers of two apart from the code, so every product that
fp32 holds is exact or the operand was not."""
import numpy as np
import pytest
import torch

from gpu_helpers import to_dev
from oracle import bf16_bits_from_f32, block4, dense
from test_gpu_linear import FORMATS, SKINNY, TILED, moe4

pytestmark = pytest.mark.gpu
SCALES = np.arange(255, dtype=np.uint8)[:, None]


def activation(fmt, e):
    """(x, x_s) of one token: 2^e, then zeros"""
    if fmt == "bf16":
        a = np.zeros((1, 32), np.float32)
        a[0, 0] = 2.0 ** e
        return to_dev(bf16_bits_from_f32(a)), None
    q = np.zeros((1, 32) if fmt == "mx8" else (1, 1, 16), np.uint8)
    q.reshape(-1)[0] = 0x38 if fmt == "mx8" else 2   # 1
    return to_dev(q), to_dev(np.full((1, 1), 127 + e, np.uint8))


def product(codes, scales, fmt, e, variant):
    q = np.zeros((len(scales), 1, 16), np.uint8)
    q[:, 0, 0] = codes
    N = -(-len(scales) // 8) * 8
    q, s = (np.resize(a, (N,) + a.shape[1:]) for a in (q, scales))
    lin = moe4.Linear(to_dev(q), to_dev(s), N=N, K=32, variant=variant)
    x, xs = activation(fmt, e)
    out = torch.empty((1, N), device="cuda")
    ws = torch.empty(moe4.moe4_linear_workspace_size(lin, 1), dtype=torch.uint8, device="cuda")
    moe4.moe4_linear_forward(lin, x, out, x_s=xs, ws=ws)
    return out.double().cpu().numpy()[0, :len(scales)], block4.values_mxfp4(q, s)[:len(scales), 0]


@pytest.mark.parametrize("variant", [SKINNY, TILED])
@pytest.mark.parametrize("fmt", FORMATS)
def test_weights(fmt, variant):
    for c in range(16):
        # 2^100 brings the smallest weights (2^-128) into the normal range, 2^-10 the largest ones
        for e in (100, 0, -10):
            got, w = product(c, SCALES, fmt, e, variant)
            want = w * 2.0 ** e
            if fmt == "bf16" or variant == SKINNY:
                want = np.where(np.abs(w) >= 2.0 ** 128, np.copysign(np.inf, w), want)
            fits = (np.abs(want) < 2.0 ** 128) | np.isinf(want)
            assert np.array_equal(got[fits], want[fits]), (c, e)
            assert np.isinf(got[~fits]).all()


@pytest.mark.parametrize("variant", [SKINNY, TILED])
def test_small_mxfp8_activations(variant):
    q = np.zeros((8, 1, 16), np.uint8)
    q[:, 0, 0] = 2
    lin = moe4.Linear(to_dev(q), to_dev(np.full((8, 1), 227, np.uint8)), N=8, K=32, variant=variant)   # 2^100
    x = np.zeros((256, 32), np.uint8)
    x[:, 0] = np.arange(256)
    for s in (0, 1, 2, 3, 4):
        xs = np.full((256, 1), s, np.uint8)
        xv = dense.mxfp8_values(x, xs)[:, 0]
        out = torch.empty((256, 8), device="cuda")
        ws = torch.empty(moe4.moe4_linear_workspace_size(lin, 256), dtype=torch.uint8, device="cuda")
        moe4.moe4_linear_forward(lin, to_dev(x), out, x_s=to_dev(xs), ws=ws)
        got = out.double().cpu().numpy()[:, 0] * 2.0 ** -100
        ok = ~np.isnan(xv)
        assert np.isnan(got[~ok]).all()
        small = ok & (np.abs(xv) < 2.0 ** -130) & (variant == SKINNY)
        assert np.array_equal(got[ok & ~small], xv[ok & ~small])
        # to the nearest multiple of 2^-133
        assert np.all(np.abs(got[small] - xv[small]) <= 2.0 ** -134)


def test_gradient():
    for s in (0, 1, 126, 252, 253, 254):
        codes = (np.arange(32) % 16).astype(np.uint8)
        q = np.tile((codes[0::2] | codes[1::2] << 4)[None, None], (8, 1, 1)).astype(np.uint8)
        lin = moe4.Linear(to_dev(q), to_dev(np.full((8, 1), s, np.uint8)), N=8, K=32)
        w = block4.values_mxfp4(q[:1], np.array([[s]], np.uint8))[0]
        up = 2.0 ** (100 if s < 2 else -10)
        dy = np.zeros((1, 8), np.float32)
        dy[0, 0] = up
        dx = torch.empty((1, 32), device="cuda")
        ws = torch.empty(moe4.moe4_linear_workspace_size(lin, 1, True), dtype=torch.uint8, device="cuda")
        moe4.moe4_linear_backward(lin, to_dev(bf16_bits_from_f32(dy)), dx, ws=ws)
        got, fits = dx.double().cpu().numpy()[0], np.abs(w) < 2.0 ** 128
        assert np.array_equal(got[fits], (w * up)[fits]), s
        assert not np.isfinite(got[~fits]).any(), s   # (0 times an infinity, from the other rows, is a NaN)
