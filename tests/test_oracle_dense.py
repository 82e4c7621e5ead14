"""Pins of the float64 definitions in oracle/dense.py: finite differences for the gradients,
exhaustive enumeration for e4m3, closed forms."""
import numpy as np
import pytest

from oracle import dense


def _diff(f, x, v, h=1e-5):
    return (f(x + h * v) - f(x - h * v)) / (2 * h)


def test_rmsnorm_is_scale_free_and_unit():
    r = np.random.default_rng(0)
    x, w = r.standard_normal((5, 24)), np.ones(24)
    s, rstd, y = dense.add_rmsnorm(x, w, 0.0)
    assert np.allclose(np.mean(y * y, 1), 1.0) and np.allclose(rstd, 1 / np.sqrt(np.mean(x * x, 1)))
    assert np.allclose(dense.add_rmsnorm(3 * x, w, 0.0)[2], y)
    assert np.allclose(dense.add_rmsnorm(x, w, 0.0, residual=2 * x)[2], y)


def test_rmsnorm_backward_against_differences():
    r = np.random.default_rng(1)
    x, w, dy = r.standard_normal((4, 16)), r.standard_normal(16), r.standard_normal((4, 16))
    dres = r.standard_normal((4, 16))
    _, rstd, _ = dense.add_rmsnorm(x, w, 1e-3)
    dx, dw = dense.add_rmsnorm_backward(dy, x, w, rstd, dres)
    vx, vw = r.standard_normal((4, 16)), r.standard_normal(16)
    fx = _diff(lambda z: np.sum(dense.add_rmsnorm(z, w, 1e-3)[2] * dy) + np.sum(z * dres), x, vx)
    fw = _diff(lambda z: np.sum(dense.add_rmsnorm(x, z, 1e-3)[2] * dy), w, vw)
    assert np.isclose(np.sum(dx * vx), fx, rtol=1e-6) and np.isclose(np.sum(dw * vw), fw, rtol=1e-6)


def _e4m3_table():
    v = []
    for c in range(127):
        e, m = c >> 3, c & 7
        v.append(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(v)


def test_e4m3_values_are_the_format():
    t = _e4m3_table()
    assert t[126] == 448.0 and t[8] == 2.0 ** -6 and t[1] == 2.0 ** -9
    codes = np.arange(128, dtype=np.uint8)
    codes[127] = 0
    got = dense.mxfp8_values(codes, np.full(4, 127, np.uint8))
    assert np.array_equal(got[:127], t)
    assert np.array_equal(dense.mxfp8_values(codes | 128, np.full(4, 129, np.uint8))[:127], -4 * t)
    assert np.isnan(dense.mxfp8_values(np.full(32, 0x7F, np.uint8), np.array([127], np.uint8))).all()


def test_mxfp8_codes_are_the_nearest_values():
    t = _e4m3_table()
    r = np.random.default_rng(2)
    x = r.standard_normal((64, 32)) * np.exp2(r.integers(-140, 120, (64, 1)).astype(float))
    q, s = dense.quantize_mxfp8(x)
    for i in range(64):
        top = np.abs(x[i]).max()
        e = int(s[i, 0]) - 127
        assert top <= 448 * 2.0 ** e and (e == -127 or top > 448 * 2.0 ** (e - 1))
        for k in range(32):
            d = np.abs(t - abs(x[i, k]) * 2.0 ** -e)
            near = np.flatnonzero(d == d.min())
            assert (q[i, k] & 127) in near
            if len(near) == 2:
                assert (q[i, k] & 127) % 2 == 0   # ties to even
            assert (q[i, k] >> 7) == int(np.signbit(x[i, k]))
    # every representable value, and the midpoints between neighbours, in a block scaled by 1
    mid = (t[:-1] + t[1:]) / 2
    for vals in (t, mid):
        for a in range(0, len(vals), 31):
            blk = np.zeros(32)
            blk[0] = 448.0
            blk[1:1 + len(vals[a:a + 31])] = vals[a:a + 31]
            q, s = dense.quantize_mxfp8(blk)
            assert s[0] == 127
            for k, v in enumerate(vals[a:a + 31]):
                want = a + k if vals is t else (a + k if (a + k) % 2 == 0 else a + k + 1)
                assert q[1 + k] == want


def test_mxfp8_special_blocks():
    x = np.zeros((5, 32))
    x[1, 3], x[2, 5], x[3, 0] = np.inf, np.nan, 448.0
    x[4, 0] = np.nextafter(448.0, 500)
    q, s = dense.quantize_mxfp8(x)
    assert s[:, 0].tolist() == [0, 255, 255, 127, 128]
    assert (q[0] == 0).all() and (q[1] == 0x7F).all() and (q[2] == 0x7F).all()
    assert q[3, 0] == 126 and q[4, 0] == 0x76


@pytest.mark.parametrize("layout", ["halves", "interleaved"])
@pytest.mark.parametrize("act", ["swiglu", "clamped"])
def test_ffn_backward_against_differences(layout, act):
    r = np.random.default_rng(3)
    T, H, I = 5, 12, 7
    x, wg, wd = r.standard_normal((T, H)), r.standard_normal((2 * I, H)), r.standard_normal((H, I))
    bg, bd, dy = r.standard_normal(2 * I), r.standard_normal(H), r.standard_normal((T, H))
    kw = dict(layout=layout, act=act, limit=2.0)

    def loss(x=x, wg=wg, wd=wd, bg=bg, bd=bd):
        return np.sum(dense.ffn_forward(x, wg, wd, b_gu=bg, b_dn=bd, **kw)["out"] * dy)

    gu = dense.ffn_forward(x, wg, wd, b_gu=bg, b_dn=bd, **kw)["gu"]
    if act == "clamped":   # the clamps are active, and no value sits at a border
        assert (np.abs(gu) > 2).any() and np.abs(np.abs(gu) - 2).min() > 1e-3
    g = dense.ffn_backward(x, gu, dy, wg, wd, **kw)
    for name, key, at in (("x", "dx", x), ("wg", "dw_gu", wg), ("wd", "dw_dn", wd),
                          ("bg", "db_gu", bg), ("bd", "db_dn", bd)):
        v = r.standard_normal(at.shape)
        want = _diff(lambda z: loss(**{name: z}), at, v, 1e-6)
        assert np.isclose(np.sum(g[key] * v), want, rtol=1e-6), key


def test_ffn_forward_by_loops():
    r = np.random.default_rng(4)
    x, wg, wd = r.standard_normal((2, 3)), r.standard_normal((4, 3)), r.standard_normal((3, 2))
    out = dense.ffn_forward(x, wg, wd, "interleaved", "swiglu", residual=x)["out"]
    for t in range(2):
        h = []
        for j in range(2):
            g, u = float(wg[2 * j] @ x[t]), float(wg[2 * j + 1] @ x[t])
            h.append(g / (1 + np.exp(-g)) * u)
        for c in range(3):
            assert np.isclose(out[t, c], x[t, c] + sum(wd[c, j] * h[j] for j in range(2)))


def test_clip():
    assert dense.grad_norm([np.array([3.0]), np.array([[4.0]])]) == 5.0
    assert dense.clip_factor(5.0, 10.0) == 1.0 and np.isclose(dense.clip_factor(5.0, 1.0), 0.2)
    assert dense.clip_factor(np.inf, 1.0) == 1.0 and dense.clip_factor(np.nan, 1.0) == 1.0
