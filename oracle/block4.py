"""A block held in 4 bits in float64 (test infrastructure only): the MXFP4 quantiser, the product with
an MXFP4 weight, the whole routed layer of a few tokens, and what stands between two blocks.
``include/moe4.h`` states what each computes; the only roundings taken here are those it states."""

import numpy as np

from .dense import ffn_activation
from .formats import mxfp4_values
from .routing import route


def quantize_mxfp4(v):
    """(blocks u8 [..., K/32, 16], scales u8 [..., K/32]) of float64 values."""
    v = np.asarray(v, np.float64)
    b = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    bad = ~np.isfinite(b).all(-1, keepdims=True)
    b = np.where(bad, 0.0, b)
    top = np.abs(b).max(-1, keepdims=True)
    # the smallest e >= -127 with top <= 7 * 2^e, by counting
    e = np.sum(top[..., 0, None] > 7.0 * np.ldexp(1.0, np.arange(-127, 128)), -1)[..., None] - 127
    q = np.abs(np.ldexp(b, -e))
    # the nearest of the eight magnitudes; on a midpoint the even code; past the last one the last
    mags = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    code = np.zeros(q.shape, np.int64)
    for c in range(7):
        mid = (mags[c] + mags[c + 1]) / 2
        code += (q > mid) | ((q == mid) & (c % 2 == 1))
    code += np.where(np.signbit(b), 8, 0)
    code = np.where(bad, 0, code).astype(np.uint8)
    scales = np.where(bad, 255, e + 127)[..., 0].astype(np.uint8)
    return code[..., 0::2] | code[..., 1::2] << 4, scales


def values_mxfp4(blocks, scales):
    """The numbers [..., K] that MXFP4 blocks [..., K/32, 16] stand for."""
    blocks, scales = np.asarray(blocks), np.asarray(scales)
    K = scales.shape[-1] * 32
    v = mxfp4_values(blocks.reshape(-1, K // 32, 16), scales.reshape(-1, K // 32))
    return v.reshape(*scales.shape[:-1], K)


def linear_forward(x, w, bias=None, residual=None):
    y = x @ w.T
    if bias is not None:
        y = y + bias
    return y if residual is None else y + residual


def linear_backward(dy, w, add=None):
    """(dx, db)"""
    dx = dy @ w
    return dx if add is None else dx + add, dy.sum(0)


def layer(x, logits, k, gu, dn, layout, act, renormalize=True, b_gu=None, b_dn=None, residual=None,
          alpha=1.702, limit=7.0, round_h=None):
    """(out [T, H], idx, weights): gu(e) and dn(e) give expert e's matrices."""
    idx, w = route(logits, k, renormalize)
    out = np.zeros((x.shape[0], np.asarray(dn(int(idx[0, 0]))).shape[0])) if x.shape[0] else x * 0.0
    for e in np.unique(idx):
        t, j = np.nonzero(idx == e)
        g = x[t] @ gu(int(e)).T
        if b_gu is not None:
            g = g + b_gu[e]
        h = ffn_activation(g, layout, act, alpha, limit)
        y = (h if round_h is None else round_h(h)) @ dn(int(e)).T
        if b_dn is not None:
            y = y + b_dn[e]
        out[t] += np.asarray(w, np.float64)[t, j][:, None] * y
    return out if residual is None else out + residual, idx, w


def join_norm(b, residual=None, res_scale=1.0, block_scale=1.0, gate=None, w_post=None, w_pre=None,
              eps=0.0, round_sum=None):
    """dict(s, ro, ri, y); ro and ri None without their norm."""
    n, ro, ri, y = b, None, None, None
    if w_post is not None:
        ro = 1.0 / np.sqrt(np.mean(b * b, 1) + eps)
        n = b * ro[:, None] * w_post
    s = block_scale * n if gate is None else block_scale * gate[:, None] * n
    if residual is not None:
        s = s + res_scale * residual
    if round_sum is not None:
        s = round_sum(s)
    if w_pre is not None:
        ri = 1.0 / np.sqrt(np.mean(s * s, 1) + eps)
        y = s * ri[:, None] * w_pre
    return {"s": s, "ro": ro, "ri": ri, "y": y}


def join_norm_backward(dy, s, b, ds=None, res_scale=1.0, block_scale=1.0, gate=None, w_post=None,
                       w_pre=None, ro=None, ri=None):
    """dict(db, dres, dgate, dw_post, dw_pre)"""
    dS = np.zeros_like(b) if ds is None else ds
    dwi = dwo = None
    if w_pre is not None:
        t = s * ri[:, None]
        p = w_pre * dy
        dS = dS + ri[:, None] * (p - t * np.mean(p * t, 1, keepdims=True))
        dwi = np.sum(dy * t, 0)
    g = np.full(b.shape[0], 1.0) if gate is None else gate
    c = (block_scale * g)[:, None]
    if w_post is not None:
        m = b * ro[:, None]
        q = w_post * dS
        along = np.sum(q * m, 1)
        db = c * ro[:, None] * (q - m * np.mean(q * m, 1, keepdims=True))
        dwo = np.sum(c * dS * m, 0)
    else:
        along = np.sum(dS * b, 1)
        db = c * dS
    return {"db": db, "dres": res_scale * dS, "dgate": block_scale * along, "dw_post": dwo,
            "dw_pre": dwi}
