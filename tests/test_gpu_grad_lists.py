"""Clipping of long lists of gradients, and at the ends of fp32's range, against float64."""
import math

import numpy as np
import pytest
import torch

from oracle import dense
from gpu_helpers import say
from test_gpu_dense import BF, F32, U32, Guarded, grads_of, rng, ueps, val, within

pytestmark = pytest.mark.gpu
moe4 = pytest.importorskip("bit_mixture_experts_amd.moe4")


def workspace(gl):
    return torch.full((moe4.moe4_grad_workspace_size(gl),), 0xFF, dtype=torch.uint8, device="cuda")


# around one launch's list and its most partial sums, and thousands of tensors of over a chunk
@pytest.mark.parametrize("n,size,dtypes", [(128, 130000, [F32]), (129, 8193, [F32, BF]), (256, 65537, [BF]),
                                           (257, 131072, [BF, F32]), (3000, 8200, [F32]), (5000, 3, [BF, F32])])
def test_clip_long_lists(n, size, dtypes):
    r = rng("long", n, size)
    few, vals = grads_of(r, [size] * 4, dtypes)
    ts = [few[i % 4].clone() for i in range(n)]
    count = [len(range(i, n, 4)) for i in range(4)]
    want = math.sqrt(sum(c * float(np.sum(v * v)) for c, v in zip(count, vals)))
    outs = [torch.zeros_like(t) for t in ts]
    gl = moe4.GradList(ts, outs)
    ws = workspace(gl)
    norm, alone = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    moe4.moe4_grad_norm(gl, alone, ws)
    ws.fill_(0xFF)
    moe4.moe4_clip_grads(gl, want / 3, norm, ws)
    assert abs(norm.item() - want) <= 2 * U32 * want and torch.equal(norm, alone)
    k = dense.clip_factor(want, want / 3)
    first = outs[:4]
    for i in range(4):
        within(val(first[i]), vals[i] * k, (ueps(few[i].dtype) + 4 * U32) * np.abs(vals[i]) * k + 1e-38, f"gradient {i}")
    bad = torch.zeros((), dtype=torch.bool, device="cuda")
    for i in range(n):
        bad |= (outs[i] != first[i % 4]).any() | (ts[i] != few[i % 4]).any()
    assert not bool(bad)


def test_clip_costs_as_much_as_its_norm_and_its_scaling():
    """One call does what moe4_grad_norm and a scaling by the norm it gives do, in about their
    time: a list's partial sums are added up a fixed number of times, not by every workgroup of
    every launch."""
    n = 1 << 16
    buf = torch.randn((n, 20), device="cuda")
    out = torch.empty_like(buf)
    gl = moe4.GradList(buf.unbind(0), out.unbind(0))
    ws, norm = workspace(gl), torch.empty(1, device="cuda")

    def whole():
        moe4.moe4_clip_grads(gl, 1.0, norm, ws)

    def parts():
        moe4.moe4_grad_norm(gl, norm, ws)
        moe4.moe4_clip_grads(gl, 1.0, norm_in=norm)

    def best(f):
        f()
        t = []
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            f()
            b.record()
            torch.cuda.synchronize()
            t.append(a.elapsed_time(b))
        return min(t)
    w, p = best(whole), best(parts)
    say(f"  {n} tensors: {w:.2f} ms in one call, {p:.2f} ms in two")
    assert w <= 2 * p


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_clip_finite_gradients_past_fp32s_norm(dtype, in_place):
    # the norm of these is 1000^1/2 * 3e38: no fp32 value, but the gradients are finite
    t = torch.full((1000,), 3e38, device="cuda").to(dtype)
    t[::2] *= -1
    v = val(t)
    o = None if in_place else Guarded((1000,), dtype)
    gl = moe4.GradList([t], None if in_place else [o.t])
    norm = torch.empty(1, device="cuda")
    moe4.moe4_clip_grads(gl, 2.0, norm, workspace(gl))
    assert math.isinf(norm.item())
    k = dense.clip_factor(dense.grad_norm([v]), 2.0)
    assert 0 < k < 1e-38
    within(val(t if in_place else o.t), v * k, (ueps(dtype) + 4 * U32) * np.abs(v) * k, "clipped")
    # an infinite norm from elsewhere says nothing of the gradients' size: unchanged
    t2 = torch.ones(100, device="cuda")
    moe4.moe4_clip_grads(moe4.GradList([t2]), 0.5, norm_in=norm)
    assert bool((t2 == 1).all())


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("max_norm", [1e-3, 1e-6, 3.0])
def test_clip_factors_below_fp32s_normal_range(dtype, max_norm):
    # max_norm / norm is a subnormal in fp32, with few bits of it left; the product is none
    r = rng("factor")
    t = torch.from_numpy((r.uniform(0.5, 1.0, 999) * 1e36).astype(np.float32)).cuda().to(dtype)
    v = val(t)
    o = Guarded((999,), dtype)
    gl = moe4.GradList([t], [o.t])
    norm = torch.empty(1, device="cuda")
    moe4.moe4_clip_grads(gl, max_norm, norm, workspace(gl))
    k = dense.clip_factor(dense.grad_norm([v]), float(np.float32(max_norm)))
    within(val(o.t), v * k, (ueps(dtype) + 4 * U32) * np.abs(v) * k, "clipped")
    o.check("clipped")
