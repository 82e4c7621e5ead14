"""The dense half of the block (norm, MXFP8, gated feed-forward block, gradient clipping) in
float64 (test infrastructure only). ``include/moe4.h`` states what each operator computes; the
only roundings taken here are those it states."""

import numpy as np

from .numerics import bf16_round_f64


def add_rmsnorm(x, weight, eps, residual=None, round_sum=None):
    """(s, rstd, y): s = round_sum(x + residual), y = s * rstd * weight. round_sum rounds to the
    residual's type (None: no rounding)."""
    s = np.asarray(x, np.float64)
    if residual is not None:
        s = s + np.asarray(residual, np.float64)
        if round_sum is not None:
            s = round_sum(s)
    rstd = 1.0 / np.sqrt(np.mean(s * s, axis=1) + eps)
    return s, rstd, s * rstd[:, None] * np.asarray(weight, np.float64)


def add_rmsnorm_backward(dy, s, weight, rstd, dres=None):
    """(dx, dweight) of add_rmsnorm for the upstream gradient dy of y."""
    n = s * rstd[:, None]
    p = dy * weight
    dx = rstd[:, None] * (p - n * np.mean(p * n, axis=1, keepdims=True))
    return dx if dres is None else dx + dres, np.sum(dy * n, axis=0)


def mxfp8_values(codes, scales):
    """The numbers that e4m3 codes [..., K] and e8m0 scales [..., K/32] stand for."""
    c = np.asarray(codes).astype(np.int64)
    e, m = (c >> 3) & 15, (c & 7).astype(np.float64)
    mag = np.where(e == 0, m * 2.0 ** -9, (8.0 + m) * np.ldexp(1.0, e - 10))
    mag = np.where((c & 127) == 127, np.nan, mag)
    s = np.asarray(scales).astype(np.int64)
    f = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    return np.where(c & 128, -mag, mag) * np.repeat(f, 32, axis=-1)


def quantize_mxfp8(v):
    """(codes u8 [..., K], scales u8 [..., K/32]) of float64 values."""
    v = np.asarray(v, np.float64)
    b = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    bad = ~np.isfinite(b).all(-1, keepdims=True)
    b = np.where(bad, 0.0, b)
    top = np.abs(b).max(-1, keepdims=True)
    # the smallest e >= -127 with top <= 448 * 2^e, by counting
    e = np.sum(top[..., 0, None] > 448.0 * np.ldexp(1.0, np.arange(-127, 128)), -1)[..., None] - 127
    q = np.ldexp(b, -e)
    # e4m3: steps of 2^-9 below 2^-6, else 1/8 of the power of two below the value
    _, ex = np.frexp(np.abs(q))
    step = np.ldexp(1.0, np.maximum(ex - 1, -6) - 3)
    r = np.rint(q / step) * step
    _, ex = np.frexp(np.abs(r))
    ex = ex - 1
    normal = np.abs(r) >= 2.0 ** -6
    m = np.where(normal, np.ldexp(np.abs(r), 3 - ex) - 8, np.abs(r) * 512).astype(np.int64)
    code = np.where(normal, (ex + 7) << 3, 0) + m + np.where(np.signbit(q), 128, 0)
    code = np.where(bad, 0x7F, code).reshape(v.shape).astype(np.uint8)
    return code, np.where(bad, 255, e + 127)[..., 0].astype(np.uint8)


def _split(gu, layout):
    I = gu.shape[-1] // 2
    return (gu[..., :I], gu[..., I:]) if layout == "halves" else (gu[..., 0::2], gu[..., 1::2])


def _join(g, u, layout):
    if layout == "halves":
        return np.concatenate([g, u], -1)
    return np.stack([g, u], -1).reshape(*g.shape[:-1], 2 * g.shape[-1])


def _sigmoid(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def ffn_activation(gu, layout, act, alpha=1.702, limit=7.0):
    g, u = _split(gu, layout)
    if act == "swiglu":
        return g * _sigmoid(g) * u
    g, u = np.where(g > limit, limit, g), np.clip(u, -limit, limit)
    return (u + 1.0) * g * _sigmoid(alpha * g)


def ffn_forward(x, w_gu, w_dn, layout, act, b_gu=None, b_dn=None, residual=None, alpha=1.702,
                limit=7.0, round_h=None):
    """dict(gu, h, out); round_h is applied to the second product's operand."""
    gu = x @ w_gu.T
    if b_gu is not None:
        gu = gu + b_gu
    h = ffn_activation(gu, layout, act, alpha, limit)
    hr = h if round_h is None else round_h(h)
    out = hr @ w_dn.T
    if b_dn is not None:
        out = out + b_dn
    return {"gu": gu, "h": hr, "out": out if residual is None else out + residual}


def ffn_backward(x, gu, dy, w_gu, w_dn, layout, act, alpha=1.702, limit=7.0, exact=True):
    """dict(dx, dw_gu, dw_dn, db_gu, db_dn); exact=False rounds dGU and h to bf16 where they are
    operands of the products that follow."""
    g, u = _split(gu, layout)
    dh = dy @ w_dn
    if act == "swiglu":
        s = _sigmoid(g)
        dg, du = dh * u * (s + g * s * (1 - s)), dh * g * s
    else:
        gc, uc = np.where(g > limit, limit, g), np.clip(u, -limit, limit)
        s = _sigmoid(alpha * gc)
        dg = np.where(g > limit, 0.0, dh * (uc + 1) * (s + alpha * gc * s * (1 - s)))
        du = np.where(np.abs(u) > limit, 0.0, dh * gc * s)
    dgu, h = _join(dg, du, layout), ffn_activation(gu, layout, act, alpha, limit)
    if not exact:
        dgu, h = bf16_round_f64(dgu), bf16_round_f64(h)
    return {"dgu": dgu, "dx": dgu @ w_gu, "dw_gu": dgu.T @ x, "dw_dn": dy.T @ h,
            "db_gu": dgu.sum(0), "db_dn": dy.sum(0)}


def grad_norm(grads):
    return float(np.sqrt(sum(float(np.sum(np.square(np.asarray(g, np.float64)))) for g in grads)))


def clip_factor(norm, max_norm):
    return min(1.0, max_norm / (norm + 1e-6)) if np.isfinite(norm) else 1.0
