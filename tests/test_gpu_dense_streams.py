"""The joined forms of the dense operators (dH cut along k with its bias sums, clipping of a list of
several launches) captured and replayed, and two of each running at once on streams of their own."""
import numpy as np
import pytest
import torch

from oracle import dense
from test_gpu_dense import BF, F32, Block, draw, rng

pytestmark = pytest.mark.gpu
moe4 = pytest.importorskip("bit_mixture_experts_amd.moe4")

T, H, I = 70, 1032, 136          # dH, dX in parts
N, SIZE = 200, 131072            # 3200 chunks of gradients, two launches


class Step:
    """A backward pass and a clipping with buffers, workspaces and inputs of their own."""

    def __init__(self, blk, key):
        self.blk = blk
        new = lambda *s, dtype=F32: torch.zeros(*s, dtype=dtype, device="cuda")   # noqa: E731
        self.dy, self.x, self.gu = new(T, H, dtype=BF), new(T, H, dtype=BF), new(T, 2 * I)
        self.out = dict(dx=new(T, H, dtype=BF), dw_gu=new(2 * I, H), dw_dn=new(H, I), db_gu=new(2 * I), db_dn=new(H))
        self.ws = blk.ws(T, True)
        self.g = new(N, SIZE)
        self.clipped = new(N, SIZE)
        self.list = moe4.GradList(self.g.unbind(0), self.clipped.unbind(0))
        self.norm = new(1)
        self.gws = torch.full((moe4.moe4_grad_workspace_size(self.list),), 0xFF, dtype=torch.uint8, device="cuda")
        self.fill(key)

    def fill(self, key):
        r = rng("streams", key)
        self.dy.copy_(draw(r, (T, H), std=0.1)[0])
        x, xv = draw(r, (T, H))
        self.x.copy_(x)
        gu = dense.ffn_forward(xv, self.blk.wg, self.blk.wd, self.blk.layout, self.blk.act, self.blk.bg)["gu"]
        self.gu.copy_(torch.from_numpy(gu.astype(np.float32)))
        gen = torch.Generator(device="cuda").manual_seed(key)
        self.g.copy_(torch.randn((N, SIZE), generator=gen, device="cuda"))

    def run(self):
        moe4.moe4_ffn_backward(self.blk.ffn, self.x, self.gu, self.dy, ws=self.ws, **self.out)
        moe4.moe4_clip_grads(self.list, 1.0, self.norm, self.gws)

    def results(self):
        return {k: v.clone() for k, v in (*self.out.items(), ("norm", self.norm), ("clipped", self.clipped))}

    def wipe(self):
        for v in (*self.out.values(), self.norm, self.clipped):
            v.fill_(float("nan"))


def same(a, b):
    for k in a:
        assert bool(torch.isfinite(a[k]).all()) and torch.equal(a[k], b[k]), k


def test_joined_forms_captured_and_replayed():
    st = Step(Block("joined", H, I, False, False, True), 1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):   # without an eager call before
        st.run()
    for key in range(2, 6):
        st.fill(key)
        st.wipe()
        g.replay()
        torch.cuda.synchronize()
        got = st.results()
        st.wipe()
        st.run()   # eager, between replays
        torch.cuda.synchronize()
        same(got, st.results())


def test_joined_forms_two_at_once():
    blk = Block("joined2", H, I, False, False, True)
    steps = [Step(blk, 11), Step(blk, 12)]
    want = []
    for st in steps:
        st.run()
        torch.cuda.synchronize()
        want.append(st.results())
        st.wipe()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s, st in zip(streams, steps):
            with torch.cuda.stream(s):
                st.run()
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for st, w in zip(steps, want):
        same(st.results(), w)
