"""Pins of the float64 definitions in oracle/block4.py: closed forms, enumeration, differences."""
import numpy as np
import pytest

from oracle import block4

MAGS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _codes(blocks):
    b = np.asarray(blocks)
    return np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], 32)


def test_mxfp4_codes_are_the_nearest_values():
    r = np.random.default_rng(0)
    x = r.standard_normal((64, 32)) * np.exp2(r.integers(-140, 120, (64, 1)).astype(float))
    q, s = block4.quantize_mxfp4(x)
    c = _codes(q)[:, 0]
    for i in range(64):
        top, e = np.abs(x[i]).max(), int(s[i, 0]) - 127
        assert top <= 7 * 2.0 ** e and (e == -127 or top > 7 * 2.0 ** (e - 1))
        for k in range(32):
            d = np.abs(MAGS - abs(x[i, k]) * 2.0 ** -e)
            assert (c[i, k] & 7) in np.flatnonzero(d == d.min())
            assert (c[i, k] >> 3) == int(np.signbit(x[i, k]))
    v = block4.values_mxfp4(q, s)
    assert np.array_equal(v, np.where(c & 8, -1, 1)[:, :] * MAGS[c & 7] * np.ldexp(1.0, s.astype(int) - 127))
    # no value is off by more than half a step: at most a quarter of it from 1 on, else a quarter
    e = np.ldexp(1.0, s.astype(int) - 127)
    assert np.all(np.abs(v - x) <= np.maximum(np.abs(x) / 4, e / 4))


def test_mxfp4_midpoints_and_ends():
    mid = (MAGS[:-1] + MAGS[1:]) / 2
    x = np.zeros((4, 32))
    x[0, :8], x[0, 8] = MAGS, 6.0
    x[1, :7], x[1, 7], x[1, 8] = mid, 7.0, -0.0
    x[2, :7] = -np.nextafter(mid, 9)
    x[2, 7] = 6.0
    x[3, 0], x[3, 1] = np.nextafter(7.0, 9), 1.0
    q, s = block4.quantize_mxfp4(x)
    c = _codes(q)[:, 0]
    assert s[:, 0].tolist() == [127, 127, 127, 128]
    assert c[0, :9].tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 7]
    assert c[1, :9].tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 8]    # ties to the even code, 7 to 6
    assert c[2, :8].tolist() == [9, 10, 11, 12, 13, 14, 15, 7]
    assert c[3, :2].tolist() == [6, 1]                         # 3.5 and a bit, and 0.5
    x[0, 3], x[1, 4] = np.inf, np.nan
    q, s = block4.quantize_mxfp4(x[:3])
    assert s[:, 0].tolist() == [255, 255, 127] and (q[:2] == 0).all()
    q, s = block4.quantize_mxfp4(np.zeros((1, 64)))
    assert (s == 0).all() and (q == 0).all()


def _diff(f, x, v, h=1e-6):
    return (f(x + h * v) - f(x - h * v)) / (2 * h)


def test_linear_by_loops_and_differences():
    r = np.random.default_rng(1)
    x, w, b, res = r.standard_normal((3, 5)), r.standard_normal((4, 5)), r.standard_normal(4), r.standard_normal((3, 4))
    y = block4.linear_forward(x, w, b, res)
    for t in range(3):
        for n in range(4):
            assert np.isclose(y[t, n], sum(x[t, i] * w[n, i] for i in range(5)) + b[n] + res[t, n])
    dy = r.standard_normal((3, 4))
    dx, db = block4.linear_backward(dy, w)
    vx, vb = r.standard_normal((3, 5)), r.standard_normal(4)
    assert np.isclose(np.sum(dx * vx), _diff(lambda z: np.sum(block4.linear_forward(z, w, b) * dy), x, vx))
    assert np.isclose(np.sum(db * vb), _diff(lambda z: np.sum(block4.linear_forward(x, w, z) * dy), b, vb))


def test_layer_by_loops():
    r = np.random.default_rng(2)
    T, E, k, H, I = 4, 5, 2, 3, 2
    x, lg = r.standard_normal((T, H)), r.standard_normal((T, E)).astype(np.float32)
    lg[1, 3] = lg[1, 1] = lg[1].max() + 1    # a tie: the lower index first
    gu, dn = r.standard_normal((E, 2 * I, H)), r.standard_normal((E, H, I))
    bg, bd = r.standard_normal((E, 2 * I)), r.standard_normal((E, H))
    out, idx, w = block4.layer(x, lg, k, lambda e: gu[e], lambda e: dn[e], "interleaved", "swiglu",
                               b_gu=bg, b_dn=bd, residual=x)
    for t in range(T):
        order = sorted(range(E), key=lambda e: (-lg[t, e], e))[:k]
        assert idx[t].tolist() == order
        p = np.exp(lg[t, order].astype(float))
        acc = x[t].copy()
        for e, q in zip(order, p / p.sum()):
            z = gu[e] @ x[t] + bg[e]
            h = [z[2 * j] / (1 + np.exp(-z[2 * j])) * z[2 * j + 1] for j in range(I)]
            acc += q * (dn[e] @ h + bd[e])
        assert np.allclose(out[t], acc)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("gated", [True, False])
def test_join_norm_against_differences(post, pre, gated):
    r = np.random.default_rng(3)
    T, H = 4, 12
    v = dict(b=r.standard_normal((T, H)), residual=r.standard_normal((T, H)),
             gate=r.standard_normal(T) if gated else None, w_post=r.standard_normal(H) if post else None,
             w_pre=r.standard_normal(H) if pre else None)
    kw = dict(res_scale=0.7, block_scale=1.3, eps=1e-3)
    dy, ds = r.standard_normal((T, H)), r.standard_normal((T, H))

    def loss(**over):
        f = block4.join_norm(**{**v, **over}, **kw)
        return np.sum(f["s"] * ds) + (np.sum(f["y"] * dy) if pre else 0.0)

    f = block4.join_norm(**v, **kw)
    g = block4.join_norm_backward(dy, f["s"], v["b"], ds, 0.7, 1.3, v["gate"], v["w_post"], v["w_pre"],
                                  f["ro"], f["ri"])
    for name, key in (("b", "db"), ("residual", "dres"), ("gate", "dgate"), ("w_post", "dw_post"),
                      ("w_pre", "dw_pre")):
        if v[name] is None:
            continue
        u = r.standard_normal(v[name].shape)
        want = _diff(lambda z: loss(**{name: z}), v[name], u)
        assert np.isclose(np.sum(g[key] * u), want, rtol=1e-5), key
    if post:
        assert np.allclose(np.mean((f["ro"][:, None] * v["b"]) ** 2, 1), 1, atol=1e-2)
