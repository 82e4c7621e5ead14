"""GPU parity of the whole routed layer for few tokens with the float64 definition in
oracle/block4.py. Tolerances count roundings: h is rounded once to bf16 (half a step, 2^-8), NF4
levels are multiplied to 2^-17, sums are fp32."""
import numpy as np
import pytest
import torch

from oracle import block4, dequantize_nf4, expand_absmax
from oracle.dense import ffn_activation
from gpu_helpers import run_layer, to_dev
from test_gpu_dense import BF, F32, RMS_BF, U32, UBF, draw, out_t, rng, within

pytestmark = pytest.mark.gpu
moe4 = pytest.importorskip("bit_mixture_experts_amd.moe4")

FMT = {"nf4": moe4.MOE4_FMT_NF4, "mx4": moe4.MOE4_FMT_MXFP4, "dq": moe4.MOE4_FMT_NF4_DQ}
LIMIT, ALPHA = 7.0, 1.702


class Stacks:
    """Random stacks on the device, and their experts' matrices in float64."""

    def __init__(self, key, fmt, E, H, I, layout="halves", act="swiglu", bias=False):
        r = rng("layer", key, fmt, E, H, I)
        self.fmt, self.E, self.H, self.I, self.layout, self.act = fmt, E, H, I, layout, act
        self.q, self.s, more = [], [], {}
        for name, N, K in (("gu", 2 * I, H), ("dn", H, I)):
            self.q.append(r.integers(0, 256, (E, N, K // 2), dtype=np.uint8))
            if fmt == "mx4":
                mid = 127 - round(np.log2(2.5 * np.sqrt(K)))
                self.s.append(r.integers(mid - 1, mid + 2, (E, N, K // 32)).astype(np.uint8))
            else:
                a = (r.uniform(0.5, 1.5, (E, N, K // 64)) * 2 / np.sqrt(K)).astype(np.float32)
                self.s.append(a)
                if fmt == "dq":
                    n = a.size
                    code, a2 = np.zeros(n, np.uint8), np.zeros(-(-n // 256), np.float32)
                    code[:] = r.integers(0, 256, n)
                    a2[:] = r.uniform(0.5, 1.0, a2.size) / np.sqrt(K)
                    off = np.array([1.5 / np.sqrt(K)], np.float32)
                    book = np.linspace(-1, 1, 256).astype(np.float32)
                    self.s[-1] = expand_absmax(code, a2, off, book).astype(np.float32).reshape(a.shape)
                    more[name + "_s2"], more[name + "_soff"], more["dq_book"] = to_dev(a2), to_dev(off), to_dev(book)
                    more[name + "_code"] = to_dev(code.reshape(a.shape))
        b = [draw(r, (E, n), std=0.2) if bias else (None, None) for n in (2 * I, H)]
        self.bias = [v for _, v in b]
        code = [more.pop("gu_code", None), more.pop("dn_code", None)]
        s = [c if c is not None else to_dev(a) for c, a in zip(code, self.s)]
        self.ex = moe4.Experts(
            FMT[fmt], to_dev(self.q[0]), s[0], to_dev(self.q[1]), s[1], E=E, H=H, I=I,
            gu_layout=moe4.MOE4_GU_HALVES if layout == "halves" else moe4.MOE4_GU_INTERLEAVED,
            act=moe4.MOE4_ACT_SWIGLU if act == "swiglu" else moe4.MOE4_ACT_SWIGLU_CLAMPED,
            gu_bias=b[0][0], dn_bias=b[1][0], act_alpha=ALPHA, act_limit=LIMIT, **more)

    def mat(self, which, e):
        q, s = self.q[which][e], self.s[which][e]
        if self.fmt == "mx4":
            return block4.values_mxfp4(q.reshape(q.shape[0], -1, 16), s)
        return np.asarray(dequantize_nf4(q.reshape(-1), s.reshape(-1)), np.float64).reshape(q.shape[0], -1)

    def ws(self, T, k):
        return torch.full((moe4.moe4_layer_decode_workspace_size(self.ex, T, k),), 0xFF, dtype=torch.uint8,
                          device="cuda")


def reference(st, xv, lg, k, renorm, res):
    """(out, idx, w, elementwise bound of fp32 outputs)"""
    out, idx, w = block4.layer(xv, lg, k, lambda e: st.mat(0, e), lambda e: st.mat(1, e), st.layout, st.act,
                               renorm, st.bias[0], st.bias[1], res, ALPHA, LIMIT)
    tol = np.zeros_like(out)
    for e in np.unique(idx):
        t, j = np.nonzero(idx == e)
        wg, wd = st.mat(0, int(e)), st.mat(1, int(e))
        gu = xv[t] @ wg.T + (st.bias[0][e] if st.bias[0] is not None else 0.0)
        dgu = (2.0 ** -17 + (st.H + 8) * U32) * (np.abs(xv[t]) @ np.abs(wg).T) + 4 * U32 * np.abs(gu)
        h = ffn_activation(gu, st.layout, st.act, ALPHA, LIMIT)
        half = st.I
        cut = ((slice(0, st.I), slice(st.I, None)) if st.layout == "halves" else (slice(0, None, 2), slice(1, None, 2)))
        g, u, dg, du = gu[:, cut[0]], gu[:, cut[1]], dgu[:, cut[0]], dgu[:, cut[1]]
        # |dh/dg| <= 1.1 |u (+ 1)| max(1, alpha), |dh/du| <= |g|
        dh = 1.9 * (np.abs(u) + 1) * dg + np.abs(g) * du + (UBF + 8 * U32) * np.abs(h)
        y = (np.abs(h) * (2.0 ** -17 + (st.I + 8) * U32) + dh) @ np.abs(wd).T
        if st.bias[1] is not None:
            y = y + 8 * U32 * np.abs(st.bias[1][e])
        tol[t] += np.asarray(w, np.float64)[t, j][:, None] * (y + 1e-5 * np.abs(h @ wd.T))
    return out, idx, w, tol + (k + 64) * U32 * np.abs(out) + 1e-30


def check(st, T, k, renorm=True, res=None, logits=None, key=0):
    r = rng("tokens", T, k, key)
    x, xv = draw(r, (T, st.H))
    lg = r.standard_normal((T, st.E)).astype(np.float32) if logits is None else logits
    rs, rv = draw(r, (T, st.H), res) if res is not None else (None, None)
    ws = st.ws(T, k)
    out, idx, w = out_t((T, st.H), F32), out_t((T, k), torch.int32), out_t((T, k), F32)
    moe4.moe4_layer_decode(st.ex, x, to_dev(lg), k, out.t, residual=rs, topk_idx=idx.t, topk_w=w.t,
                           renormalize=renorm, ws=ws)
    wo, wi, ww, tol = reference(st, xv, lg, k, renorm, rv)
    assert np.array_equal(idx.t.cpu().numpy(), wi)
    gw = w.t.double().cpu().numpy()
    assert np.all(np.abs(gw - ww) <= 1e-5 * ww)
    got = out.t.double().cpu().numpy()
    within(got, wo, tol, f"out {st.fmt} T {T}")
    base = rv if rv is not None else 0.0
    rel = np.linalg.norm(got - wo, axis=1) / np.linalg.norm(wo - base, axis=1)
    assert rel.max() <= 2 * RMS_BF, rel.max()
    # bf16 is the same sum rounded once; without the routing's outputs the same bits
    o16 = out_t((T, st.H), BF)
    moe4.moe4_layer_decode(st.ex, x, to_dev(lg), k, o16.t, residual=rs, renormalize=renorm, ws=ws)
    assert torch.equal(o16.t, out.t.to(BF))
    for g in (out, idx, w, o16):
        g.check("layer")
    return x, lg, out.t


CASES = [("nf4", 8, 2, 256, 512, "halves", "swiglu", False), ("mx4", 8, 2, 256, 512, "interleaved", "clamped", True),
         ("dq", 8, 2, 256, 512, "halves", "swiglu", False), ("mx4", 5, 3, 32, 32, "halves", "swiglu", False),
         ("nf4", 3, 3, 64, 64, "interleaved", "clamped", True), ("dq", 4, 1, 64, 128, "interleaved", "swiglu", True),
         ("nf4", 16, 4, 832, 320, "halves", "clamped", False), ("mx4", 32, 4, 2880, 2880, "interleaved", "clamped", True),
         ("nf4", 128, 8, 2048, 768, "halves", "swiglu", False), ("mx4", 300, 16, 96, 160, "halves", "clamped", True),
         ("nf4", 1024, 3, 128, 64, "halves", "swiglu", False), ("dq", 140, 8, 2048, 768, "halves", "swiglu", False)]


@pytest.mark.parametrize("T", [1, 2, 7, 9, 16, 32])
@pytest.mark.parametrize("fmt,E,k,H,I,layout,act,bias", CASES)
def test_layer_decode(fmt, E, k, H, I, layout, act, bias, T):
    if T * k > moe4.MOE4_LAYER_MOST_SLOTS or (H * I > 1 << 20 and T in (2, 7, 32)):
        pytest.skip("beyond the slots of one call, or a wide expert at a size that narrow ones cover")
    check(Stacks("a", fmt, E, H, I, layout, act, bias), T, k, renorm=T != 7, res=(None, BF, F32)[T % 3])


# enough units of work that the second launch cuts its panels: runs of 2, 3 and 4 steps, few and many
# units to a panel (parts of one panel by many workgroups, many panels to one), groups of tokens; and some
# that are just too few
@pytest.mark.parametrize("fmt,T,E,k,H,I,bias", [
    ("nf4", 32, 24, 8, 1088, 320, True), ("nf4", 9, 64, 8, 2112, 832, False), ("nf4", 32, 128, 16, 512, 64, False),
    ("nf4", 32, 128, 16, 256, 64, False), ("nf4", 4, 128, 8, 2048, 768, True), ("mx4", 32, 40, 16, 416, 1312, True),
    ("mx4", 8, 32, 4, 2880, 2080, True), ("mx4", 17, 300, 30, 416, 32, False), ("mx4", 32, 16, 16, 416, 1024, True),
    ("mx4", 32, 40, 16, 160, 1312, True), ("dq", 25, 12, 6, 1024, 1088, True), ("dq", 32, 16, 16, 512, 448, False),
    ("dq", 10, 64, 8, 1664, 448, False)])
def test_layer_decode_many_units(fmt, T, E, k, H, I, bias):
    assert (H // 16) * T * k >= 4096
    st = Stacks("units", fmt, E, H, I, "interleaved" if bias else "halves", "clamped" if bias else "swiglu", bias)
    x, lg, out = check(st, T, k, res=(BF, F32, None)[T % 3])
    if T % 3 == 2:   # (without a residual) the same bits again, whoever came last
        ws = st.ws(T, k)
        for _ in range(3):
            again = torch.full_like(out, float("nan"))
            moe4.moe4_layer_decode(st.ex, x, to_dev(lg), k, again, ws=ws)
            assert torch.equal(again, out)


def test_many_units_of_one_expert_and_of_all():
    for E, k in ((1, 1), (16, 16)):
        st = Stacks("all", "mx4", E, 2080, 2080)
        check(st, 32, k)


def test_many_units_captured_and_two_at_once():
    st = Stacks("cap", "nf4", 48, 1600, 256)
    T, k = 16, 8
    buf = [dict(x=torch.zeros((T, 1600), dtype=BF, device="cuda"), lg=torch.zeros((T, 48), device="cuda"),
                out=torch.zeros((T, 1600), dtype=BF, device="cuda"), ws=st.ws(T, k)) for _ in range(2)]

    def fill(b, key):
        r = rng("cap fill", key)
        b["x"].copy_(draw(r, (T, 1600))[0])
        b["lg"].copy_(to_dev(r.standard_normal((T, 48)).astype(np.float32)))
        b["out"].fill_(float("nan"))

    def run(b, stream=None):
        moe4.moe4_layer_decode(st.ex, b["x"], b["lg"], k, b["out"], ws=b["ws"], stream=stream)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(buf[0])
    want = []
    for key in range(3):
        fill(buf[0], key)
        g.replay()
        torch.cuda.synchronize()
        got = buf[0]["out"].clone()
        buf[0]["out"].fill_(float("nan"))
        run(buf[0])
        assert torch.equal(got, buf[0]["out"]) and bool(torch.isfinite(got).all())
    for i in (0, 1):
        fill(buf[i], 10 + i)
        run(buf[i])
        want.append(buf[i]["out"].clone())
        buf[i]["out"].fill_(float("nan"))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for i, s in enumerate(streams):
            run(buf[i], s)
    torch.cuda.synchronize()
    assert all(torch.equal(buf[i]["out"], want[i]) for i in (0, 1))


@pytest.mark.parametrize("fmt", ["nf4", "mx4", "dq"])
def test_every_token_takes_the_same_experts(fmt):
    # rows of one expert over several passes of 8; every expert chosen (k = E); one expert
    for E, k, T in ((8, 2, 32), (4, 4, 31), (1, 1, 17), (16, 16, 32)):
        st = Stacks("b", fmt, E, 192, 128)
        lg = np.tile(rng("same", E).standard_normal(E).astype(np.float32), (T, 1))
        check(st, T, k, logits=lg)


def test_ties_infinities_and_zeros_in_the_logits():
    st = Stacks("c", "nf4", 70, 128, 64)
    r = rng("ties")
    lg = r.integers(-2, 3, (9, 70)).astype(np.float32)     # ties everywhere: the lower index first
    lg[0] = 0.0
    lg[1, ::2] = -0.0
    lg[1, 1::2] = 0.0
    lg[2, 5:] = -np.inf
    lg[3] = np.linspace(-3e38, 3e38, 70, dtype=np.float32)
    lg[4, 3], lg[4, 60] = 1e-45, -1e-45
    check(st, 9, 5, logits=lg)
    check(st, 9, 5, logits=lg, renorm=False)


def test_matches_the_separate_calls():
    # MXFP4, whose weights are exact on both ways: the same routing, and outputs of the same h
    st = Stacks("d", "mx4", 16, 512, 256, "interleaved", "clamped", True)
    x, lg, out = check(st, 13, 4)
    r = run_layer(st.ex, x, to_dev(lg), 4)
    rms = float(r["out32"].double().square().mean().sqrt())
    # a value of h on a rounding's border takes its other neighbour: a few of them per row
    assert float((r["out32"] - out).abs().max()) <= 1e-2 * rms


def test_nan_stays_with_its_token():
    for fmt in ("nf4", "mx4"):
        st = Stacks("e", fmt, 6, 128, 96 if fmt == "mx4" else 128)
        r = rng("nan", fmt)
        x, _ = draw(r, (12, 128))
        lg = to_dev(r.standard_normal((12, 6)).astype(np.float32))
        out, want = torch.empty((12, 128), device="cuda"), torch.empty((12, 128), device="cuda")
        ws = st.ws(12, 2)
        moe4.moe4_layer_decode(st.ex, x, lg, 2, want, ws=ws)
        x[3, 17], x[8, 0] = float("nan"), float("inf")
        moe4.moe4_layer_decode(st.ex, x, lg, 2, out, ws=ws)
        rest = [t for t in range(12) if t not in (3, 8)]
        assert bool(torch.isnan(out[3]).all()) and not bool(torch.isfinite(out[8]).all())
        assert torch.equal(out[rest], want[rest])


def test_nan_logits_choose_distinct_experts():
    st = Stacks("f", "nf4", 9, 64, 64)
    lg = torch.full((3, 9), float("nan"), device="cuda")
    lg[1, 4] = 1.0
    x, _ = draw(rng("nanlog"), (3, 64))
    idx, out = torch.empty((3, 4), dtype=torch.int32, device="cuda"), torch.empty((3, 64), dtype=BF, device="cuda")
    moe4.moe4_layer_decode(st.ex, x, lg, 4, out, topk_idx=idx, ws=st.ws(3, 4))
    for row in idx.cpu().tolist():
        assert len(set(row)) == 4 and all(0 <= e < 9 for e in row)
    assert int(idx[1, 0]) == 4


def test_in_place_and_scale_255():
    st = Stacks("g", "mx4", 4, 64, 64)
    r = rng("place")
    x, _ = draw(r, (5, 64))
    lg = to_dev(r.standard_normal((5, 4)).astype(np.float32))
    res, _ = draw(r, (5, 64))
    ws = st.ws(5, 2)
    want = torch.empty((5, 64), dtype=BF, device="cuda")
    moe4.moe4_layer_decode(st.ex, x, lg, 2, want, residual=res, ws=ws)
    for target in ("res", "x"):
        a, b = x.clone(), res.clone()
        o = b if target == "res" else a
        moe4.moe4_layer_decode(st.ex, a, lg, 2, o, residual=b, ws=ws)
        assert torch.equal(o, want)
    # an e8m0 NaN in one output row of every expert: that column alone
    st.ex.tensors[3][:, 7, 1] = 255
    out = torch.empty((5, 64), device="cuda")
    moe4.moe4_layer_decode(st.ex, x, lg, 2, out, ws=ws)
    assert bool(torch.isnan(out[:, 7]).all())
    assert bool(torch.isfinite(torch.cat((out[:, :7], out[:, 8:]), 1)).all())


def test_captured_replayed_and_two_at_once():
    st = Stacks("h", "nf4", 32, 512, 256)
    steps = []
    for key in range(2):
        x, lg = torch.zeros((6, 512), dtype=BF, device="cuda"), torch.zeros((6, 32), device="cuda")
        steps.append((x, lg, torch.zeros((6, 512), dtype=BF, device="cuda"), st.ws(6, 4)))

    def fill(i, key):
        r = rng("fill", key)
        steps[i][0].copy_(draw(r, (6, 512))[0])
        steps[i][1].copy_(to_dev(r.standard_normal((6, 32)).astype(np.float32)))

    def run(i, stream=None):
        x, lg, out, ws = steps[i]
        moe4.moe4_layer_decode(st.ex, x, lg, 4, out, ws=ws, stream=stream)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(0)
    for key in range(4):
        fill(0, key)
        steps[0][2].fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        got = steps[0][2].clone()
        steps[0][2].fill_(float("nan"))
        run(0)
        torch.cuda.synchronize()
        assert torch.equal(got, steps[0][2]) and bool(torch.isfinite(got).all())
    fill(1, 9)
    want = []
    for i in (0, 1):
        run(i)
        torch.cuda.synchronize()
        want.append(steps[i][2].clone())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for i, s in enumerate(streams):
            s.wait_stream(torch.cuda.current_stream())
            run(i, s)
    torch.cuda.synchronize()
    for i in (0, 1):
        assert torch.equal(steps[i][2], want[i])


def test_refusals():
    st = Stacks("i", "nf4", 8, 64, 64)
    e = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype, device="cuda")   # noqa: E731
    ws = st.ws(2, 2)
    ok = dict(ws=ws)
    moe4.moe4_layer_decode(st.ex, e(0, 64), e(0, 8, dtype=F32), 2, e(0, 64), **ok)
    for x, lg, k, out, kw, err in (
            (e(33, 64), e(33, 8, dtype=F32), 2, e(33, 64), ok, moe4.Moe4Error),
            (e(2, 64), e(2, 8, dtype=F32), 9, e(2, 64), ok, moe4.Moe4Error),
            (e(2, 64), e(2, 8, dtype=F32), 0, e(2, 64), ok, moe4.Moe4Error),
            (e(2, 64), e(2, 7, dtype=F32), 2, e(2, 64), ok, ValueError),
            (e(2, 32), e(2, 8, dtype=F32), 2, e(2, 64), ok, ValueError),
            (e(2, 64), e(2, 8), 2, e(2, 64), ok, TypeError),
            (e(2, 64), e(2, 8, dtype=F32), 2, e(3, 64), ok, ValueError),
            (e(2, 64), e(2, 8, dtype=F32), 2, e(2, 64), {}, moe4.Moe4Error),
            (e(2, 64), e(2, 8, dtype=F32), 2, e(2, 64), dict(ws=ws[:64]), moe4.Moe4Error),
            (e(2, 64).cpu(), e(2, 8, dtype=F32), 2, e(2, 64), ok, TypeError)):
        with pytest.raises(err):
            moe4.moe4_layer_decode(st.ex, x, lg, k, out, **kw)
    with pytest.raises(moe4.Moe4Error):
        moe4.moe4_layer_decode(st.ex.with_variant(moe4.MOE4_VARIANT_TILED), e(2, 64), e(2, 8, dtype=F32), 2,
                               e(2, 64), **ok)
