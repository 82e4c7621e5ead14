"""Infinite activations through the routed layer for few tokens: what the definition gives, infinities
of its sign and, behind the clamped activation, finite numbers, and not the NaNs of an infinity times
one part of a weight."""
import numpy as np
import pytest
import torch

from gpu_helpers import to_dev
from test_gpu_dense import BF, U32, UBF, draw, rng
from test_gpu_layer_decode import ALPHA, LIMIT, Stacks, moe4

pytestmark = pytest.mark.gpu


def set_codes(st, fmt, at):
    """Every weight that meets activation `at`, and each row of the down matrices whole, of one sign and
    not zero: gates and ups positive, down rows positive, negative, positive, ..."""
    r = rng("signs", fmt)
    pos, neg = (np.arange(8, 16), np.arange(0, 7)) if fmt != "mx4" else (np.arange(1, 8), np.arange(9, 16))
    gu, dn = st.q
    every = np.resize(pos, gu.shape[:2])   # every positive level
    gu[:, :, at // 2] = gu[:, :, at // 2] & (0x0F if at & 1 else 0xF0) | every << (4 if at & 1 else 0)
    for n in range(st.H):
        v = r.choice(neg if n & 1 else pos, (st.E, st.I))
        dn[:, n] = v[:, 0::2] | v[:, 1::2] << 4
    st.ex.tensors[0].copy_(to_dev(gu))
    st.ex.tensors[2].copy_(to_dev(dn))


# the second shape has units enough that the second launch cuts its panels
@pytest.mark.parametrize("T,E,k,H,I", [(5, 2, 2, 128, 192), (32, 16, 16, 512, 448)])
@pytest.mark.parametrize("act", ["swiglu", "clamped"])
@pytest.mark.parametrize("fmt", ["nf4", "dq", "mx4"])
def test_infinite_activation(fmt, act, T, E, k, H, I):
    at, t = 37, 2
    st = Stacks("inf", fmt, E, H, I, "halves", act)
    set_codes(st, fmt, at)
    x, xv = draw(rng("inf x"), (T, H))
    lg = to_dev(rng("inf lg").standard_normal((T, E)).astype(np.float32))
    run = lambda out, w=None: moe4.moe4_layer_decode(st.ex, x, lg, k, out, topk_w=w, ws=st.ws(T, k))   # noqa: E731
    want, out = (torch.empty((T, H), device="cuda") for _ in range(2))
    w = torch.empty((T, k), device="cuda")
    run(want)
    x[t, at] = float("inf")
    run(out, w)
    rest = [i for i in range(T) if i != t]
    assert torch.equal(out[rest], want[rest])
    got = out[t].double().cpu().numpy()
    if act == "swiglu":   # gates, ups and so h are +inf, each output of its row's sign
        assert np.array_equal(got, np.where(np.arange(H) & 1, -np.inf, np.inf))
        return
    # the clamp takes gates and ups to its limit, so all h are one number
    h = (LIMIT + 1) * LIMIT / (1 + np.exp(-ALPHA * LIMIT))
    tw = np.zeros(E)
    idx = np.argsort(-lg[t].cpu().numpy(), kind="stable")[:k]
    tw[idx] = w[t].double().cpu().numpy()
    y = sum(tw[e] * h * st.mat(1, e).sum(1) for e in range(E))
    mag = sum(tw[e] * h * np.abs(st.mat(1, e)).sum(1) for e in range(E))
    # w h rounded to bf16 (half a step), a level to 2^-16, fp32 sums over experts and I, sigmoid to 8 steps
    assert np.all(np.abs(got - y) <= (UBF + 2.0 ** -16 + (k * I + 24) * U32) * mag)


def test_negative_infinity_and_zero_weights_give_what_the_formula_gives():
    # -inf gates: silu(-inf) = -inf * 0, a NaN; a zero weight times an infinity is one too
    for fmt, zero in (("nf4", 7), ("mx4", 0)):
        st = Stacks("zero", fmt, 1, 64, 64)
        set_codes(st, fmt, 0)
        x, _ = draw(rng("zero x"), (2, 64))
        lg, out = torch.zeros((2, 1), device="cuda"), torch.empty((2, 64), dtype=BF, device="cuda")
        x[1, 0] = float("-inf")
        moe4.moe4_layer_decode(st.ex, x, lg, 1, out, ws=st.ws(2, 1))
        assert bool(out[1].isnan().all()) and bool(out[0].isfinite().all())
        x[1, 0] = float("inf")
        st.ex.tensors[0][:, 3, 0] = st.ex.tensors[0][:, 3, 0] & 0xF0 | zero
        moe4.moe4_layer_decode(st.ex, x, lg, 1, out, ws=st.ws(2, 1))
        assert bool(out[1].isnan().all()) and bool(out[0].isfinite().all())
