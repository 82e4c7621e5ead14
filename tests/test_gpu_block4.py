"""The operators of a block held in 4 bits, run together as they are used: a decode step (projection,
join, router, routed layer, join in MXFP4, projection) and a training pair (join and frozen projection
with their gradients). Each step is held against the float64 definition on the values that the step
before it passed on; a row of values rounded to bf16 is off by 2^-8 / sqrt(3) of it in the root mean
square, with a factor of two for the spread of one row, and fp32 sums by less than 1e-5."""
import math

import numpy as np
import pytest
import torch

from oracle import block4
from gpu_helpers import to_dev
from test_gpu_dense import BF, F32, RMS_BF, draw, rng, row_norm, val
from test_gpu_layer_decode import ALPHA, LIMIT, Stacks
from test_gpu_linear import Weight

pytestmark = pytest.mark.gpu
moe4 = pytest.importorskip("bit_mixture_experts_amd.moe4")

EPS = 1e-6
ONE = 2 * RMS_BF + 1e-5   # a row rounded once to bf16


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8, device="cuda")


class DecodeStep:
    """stream, x (bf16) -> the stream after the block and the next projection (f32)"""

    def __init__(self, fmt, T, H, I, E, k, N):
        r = rng("step", fmt, T, H)
        self.T, self.H, self.k = T, H, k
        self.st = Stacks("step", fmt, E, H, I, "interleaved", "clamped", True)
        self.proj, self.next = Weight("proj", H, H, True), Weight("next", N, H)
        self.w = [draw(r, (H,), std=0.3) for _ in range(4)]
        self.wr, self.wrv = draw(r, (E, H), std=1 / math.sqrt(H))
        z = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype, device="cuda")   # noqa: E731
        self.t = dict(x=z(T, H), stream=z(T, H), xq=u8(T, H // 32, 16), xs=u8(T, H // 32), b=z(T, H), s=z(T, H), n=z(T, H),
                      lg=z(T, E, dtype=F32), o=z(T, H), s2=z(T, H), n2=z(T, H), q=u8(T, H // 32, 16), qs=u8(T, H // 32),
                      y=z(T, N, dtype=F32))
        self.ws = [self.proj.ws(T), self.st.ws(T, k), self.next.ws(T)]

    def fill(self, key):
        r = rng("fill", key)
        for n in ("x", "stream"):
            self.t[n].copy_(draw(r, (self.T, self.H))[0])

    def run(self, stream=None):
        t, w, kw = self.t, [a for a, _ in self.w], dict(stream=stream)
        moe4.moe4_quantize_mxfp4(t["x"], t["xq"], t["xs"], **kw)
        moe4.moe4_linear_forward(self.proj.lin, t["xq"], t["b"], x_s=t["xs"], ws=self.ws[0], **kw)
        moe4.moe4_join_norm(t["b"], w[1], EPS, residual=t["stream"], block_scale=0.5, w_post=w[0], sum_out=t["s"],
                            out=t["n"], **kw)
        moe4.moe4_router_logits(t["n"], self.wr, t["lg"], **kw)
        moe4.moe4_layer_decode(self.st.ex, t["n"], t["lg"], self.k, t["o"], ws=self.ws[1], **kw)
        moe4.moe4_join_norm(t["o"], w[3], EPS, residual=t["s"], block_scale=0.5, w_post=w[2], sum_out=t["s2"], out=t["n2"],
                            out_q=t["q"], out_s=t["qs"], **kw)
        moe4.moe4_linear_forward(self.next.lin, t["q"], t["y"], x_s=t["qs"], ws=self.ws[2], **kw)

    def check(self):
        t, w, st = self.t, [v for _, v in self.w], self.st
        n = {a: t[a].cpu().numpy() for a in ("xq", "xs", "q", "qs", "lg")}
        q, s = block4.quantize_mxfp4(val(t["x"]))[:2]
        assert np.array_equal(n["xq"].reshape(self.T, -1), q.reshape(self.T, -1)) and np.array_equal(n["xs"], s)
        x = block4.values_mxfp4(n["xq"], n["xs"])
        row_norm(val(t["b"]), block4.linear_forward(x, self.proj.w, self.proj.bias), ONE, "projection")
        j = block4.join_norm(val(t["b"]), val(t["stream"]), block_scale=0.5, w_post=w[0], w_pre=w[1], eps=EPS)
        row_norm(val(t["s"]), j["s"], ONE, "stream")
        j = block4.join_norm(val(t["s"]), w_pre=w[1], eps=EPS)   # (the row that the second norm sees)
        row_norm(val(t["n"]), j["y"], ONE, "norm")
        row_norm(n["lg"].astype(np.float64), val(t["n"]) @ self.wrv.T, 1e-5, "logits")
        o = block4.layer(val(t["n"]), n["lg"], self.k, lambda e: st.mat(0, e), lambda e: st.mat(1, e), st.layout, st.act,
                         True, st.bias[0], st.bias[1], None, ALPHA, LIMIT)[0]
        row_norm(val(t["o"]), o, 2 * ONE, "layer (h and out rounded)")
        j = block4.join_norm(val(t["o"]), val(t["s"]), block_scale=0.5, w_post=w[2], w_pre=w[3], eps=EPS)
        row_norm(val(t["s2"]), j["s"], ONE, "second stream")
        j = block4.join_norm(val(t["s2"]), w_pre=w[3], eps=EPS)
        row_norm(val(t["n2"]), j["y"], ONE, "second norm")
        v = block4.values_mxfp4(n["q"], n["qs"])
        step = np.maximum(np.abs(j["y"]), np.repeat(np.ldexp(1.0, n["qs"].astype(int) - 127), 32, 1))
        assert np.all(np.abs(v - j["y"]) <= (0.25 + 1e-5) * step)   # half a step of e2m1, 1/4 of the value or of the scale
        row_norm(val(t["y"]), block4.linear_forward(v, self.next.w), 1e-5, "next projection")


STEPS = [("mx4", 1, 256, 288, 12, 3, 136), ("nf4", 8, 512, 320, 16, 4, 264), ("dq", 13, 192, 128, 9, 9, 72),
         ("mx4", 32, 2080, 544, 16, 4, 520)]


@pytest.mark.parametrize("fmt,T,H,I,E,k,N", STEPS)
def test_decode_step(fmt, T, H, I, E, k, N):
    d = DecodeStep(fmt, T, H, I, E, k, N)
    d.fill(0)
    d.run()
    d.check()


@pytest.mark.parametrize("fmt,T,H,I,E,k,N", STEPS[1:2] + STEPS[3:])
def test_decode_step_captured_and_two_at_once(fmt, T, H, I, E, k, N):
    d, other = DecodeStep(fmt, T, H, I, E, k, N), DecodeStep(fmt, T, H, I, E, k, N)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d.run()
    for key in range(3):
        for a in (d, other):
            a.fill(key)
        g.replay()
        other.run()     # eager, of the same values, on the same weights' copies
        torch.cuda.synchronize()
        assert all(torch.equal(d.t[n], other.t[n]) for n in d.t)
    d.check()
    # two steps at once, on streams of their own
    d.fill(7), other.fill(8)
    want = []
    for a in (d, other):
        a.run()
        want.append({n: v.clone() for n, v in a.t.items()})
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for a, s in zip((d, other), streams):
            a.run(s)
    torch.cuda.synchronize()
    for a, w in zip((d, other), want):
        assert all(torch.equal(a.t[n], w[n]) for n in a.t)


class TrainPair:
    """join (gate, both norms) -> frozen projection, and back"""

    def __init__(self, T, H, N):
        r = rng("train", T, H, N)
        self.T, self.H, self.N = T, H, N
        self.wt = Weight("train", N, H)
        (self.wo, self.wov), (self.wi, self.wiv) = (draw(r, (H,)) for _ in range(2))
        z = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype, device="cuda")   # noqa: E731
        self.t = dict(b=z(T, H), res=z(T, H), gate=z(T, dtype=F32), g=z(T, N), s=z(T, H), n=z(T, H), ro=z(T, dtype=F32),
                      ri=z(T, dtype=F32), y=z(T, N), dn=z(T, H), db=z(T, H), dres=z(T, H), dgate=z(T, dtype=F32),
                      dwo=z(H, dtype=F32), dwi=z(H, dtype=F32), dbias=z(N, dtype=F32))
        self.ws = [self.wt.ws(T), self.wt.ws(T, True),
                   torch.empty(moe4.moe4_join_norm_workspace_size(T, H), dtype=torch.uint8, device="cuda")]

    def fill(self, key):
        r = rng("fill", key)
        for n in ("b", "res", "g"):
            self.t[n].copy_(draw(r, tuple(self.t[n].shape))[0])
        self.t["gate"].copy_(to_dev(r.uniform(0.2, 1.0, self.T).astype(np.float32)))

    def run(self):
        t = self.t
        kw = dict(res_scale=0.75, block_scale=0.5, gate=t["gate"], w_post=self.wo)
        moe4.moe4_join_norm(t["b"], self.wi, EPS, residual=t["res"], sum_out=t["s"], out=t["n"], rstd_post=t["ro"],
                            rstd_pre=t["ri"], **kw)
        moe4.moe4_linear_forward(self.wt.lin, t["n"], t["y"], ws=self.ws[0])
        moe4.moe4_linear_backward(self.wt.lin, t["g"], t["dn"], db=t["dbias"], ws=self.ws[1])
        moe4.moe4_join_norm_backward(t["dn"], t["s"], t["b"], self.wi, t["ri"], t["db"], dres=t["dres"], rstd_post=t["ro"],
                                     dgate=t["dgate"], dw_post=t["dwo"], dw_pre=t["dwi"], ws=self.ws[2], **kw)

    def loss(self, b, res, gate, wo, wi):
        j = block4.join_norm(b, res, 0.75, 0.5, gate, wo, wi, EPS)
        return np.sum(block4.linear_forward(j["y"], self.wt.w) * val(self.t["g"]))


@pytest.mark.parametrize("T,H,N", [(33, 256, 136), (130, 1056, 264)])
def test_training_pair(T, H, N):
    p = TrainPair(T, H, N)
    p.fill(0)
    p.run()
    t = {n: val(a) for n, a in p.t.items()}
    # against the formulas, on the values that were passed on
    row_norm(t["y"], block4.linear_forward(t["n"], p.wt.w), ONE, "y")
    dn, dbias = block4.linear_backward(t["g"], p.wt.w)
    row_norm(t["dn"], dn, ONE, "dn")
    assert np.linalg.norm(t["dbias"] - dbias) <= 1e-5 * np.linalg.norm(dbias)
    w = block4.join_norm_backward(t["dn"], t["s"], t["b"], None, 0.75, 0.5, t["gate"], p.wov, p.wiv, t["ro"], t["ri"])
    row_norm(t["db"], w["db"], ONE, "db")
    row_norm(t["dres"], w["dres"], ONE, "dres")
    for n, a in (("dgate", "dgate"), ("dwo", "dw_post"), ("dwi", "dw_pre")):
        assert np.linalg.norm(t[n] - w[a]) <= 1e-4 * np.linalg.norm(w[a]), n
    # and against differences of the whole in float64: s and dn are rounded to bf16 on the way (s twice
    # in effect, in the forward and as the backward's operand), db and dres once more
    r = rng("dir")
    at = [t["b"], t["res"], t["gate"], p.wov, p.wiv]
    for i, got in enumerate((t["db"], t["dres"], t["dgate"], t["dwo"], t["dwi"])):
        v = r.standard_normal(at[i].shape)
        h = 1e-5
        up, dn_ = [a.copy() for a in at], [a.copy() for a in at]
        up[i] = up[i] + h * v
        dn_[i] = dn_[i] - h * v
        diff = (p.loss(*up) - p.loss(*dn_)) / (2 * h)
        # (in a random direction errors add as the root of their squares: 4 roundings, times 4)
        assert abs(np.sum(got * v) - diff) <= 4 * 4 * RMS_BF * np.linalg.norm(got) + 1e-6 * abs(diff), i


def test_training_pair_captured():
    p, other = TrainPair(130, 1056, 264), TrainPair(130, 1056, 264)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.run()
    for key in range(4):
        for a in (p, other):
            a.fill(key)
        g.replay()
        other.run()
        torch.cuda.synchronize()
        assert all(torch.equal(p.t[n], other.t[n]) for n in p.t)
