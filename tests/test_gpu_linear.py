"""GPU parity of the dense product with an MXFP4 weight, and of its gradients, with the float64
definition in oracle/block4.py.

Tolerances count roundings. Operands are exact (bf16 holds an e2m1 or e4m3 value times its power of
two), so an fp32 output is off by the sum alone: n terms, bias, residual, each addition by at most
2^-24 of the magnitudes' sum. Products of two e2m1 values are multiples of 1/4 up to 36, which the
scaled matrix instruction keeps; with e4m3 it keeps the 32 products of a block each to 2^-16 of the
largest. A bf16 output is rounded once more, by 2^-8 of its value."""
import numpy as np
import pytest
import torch

from oracle import bf16_bits_from_f32, bf16_bits_to_f64, block4, dense
from gpu_helpers import to_dev
from test_gpu_dense import BF, F32, U32, draw, out_t, rng, ueps, val, within

pytestmark = pytest.mark.gpu
moe4 = pytest.importorskip("bit_mixture_experts_amd.moe4")

SKINNY, TILED = moe4.MOE4_VARIANT_SKINNY, moe4.MOE4_VARIANT_TILED
FORMATS = ["bf16", "mx8", "mx4"]


class Weight:
    def __init__(self, key, N, K, bias=False):
        r = rng("lin", key, N, K)
        self.N, self.K = N, K
        q = r.integers(0, 256, (N, K // 32, 16), dtype=np.uint8)
        mid = 127 - round(np.log2(2.5 * np.sqrt(K)))
        s = r.integers(mid - 1, mid + 2, (N, K // 32)).astype(np.uint8)
        b, self.bias = draw(r, (N,), std=0.3) if bias else (None, None)
        self.q, self.s = q, s
        self.w = block4.values_mxfp4(q, s)
        self.lin = moe4.Linear(to_dev(q), to_dev(s), N=N, K=K, bias=b)

    def ws(self, T, backward=False):   # NaNs wherever it is read before it is written
        return torch.full((moe4.moe4_linear_workspace_size(self.lin, T, backward),), 0xFF, dtype=torch.uint8,
                          device="cuda")


def tokens(fmt, T, K, key=0):
    """(x, x_s, values)"""
    x, xv = draw(rng("lin x", key, T, K), (T, K))
    if fmt == "bf16":
        return x, None, xv
    if fmt == "mx8":
        q, s = dense.quantize_mxfp8(xv)
        return to_dev(q), to_dev(s), dense.mxfp8_values(q, s)
    q, s = block4.quantize_mxfp4(xv)[:2]
    q = q.reshape(T, K // 32, 16)
    return to_dev(q), to_dev(s), block4.values_mxfp4(q, s)


def check(wt, fmt, T, variant, out_dtype, res_dtype, key=0):
    x, xs, xv = tokens(fmt, T, wt.K, key)
    res, rv = draw(rng("res", T, wt.N), (T, wt.N), res_dtype) if res_dtype is not None else (None, None)
    out = out_t((T, wt.N), out_dtype)
    moe4.moe4_linear_forward(wt.lin.with_variant(variant), x, out.t, x_s=xs, residual=res, ws=wt.ws(T))
    used = moe4.moe4_last_variant()
    want = block4.linear_forward(xv, wt.w, wt.bias, rv)
    mag = np.abs(xv) @ np.abs(wt.w).T + (0 if wt.bias is None else np.abs(wt.bias)) + (0 if rv is None else np.abs(rv))
    unit = 32 * 2.0 ** -16 if fmt == "mx8" and used == TILED else 0.0
    u = 0.0 if out_dtype == F32 else ueps(out_dtype)
    err = ((wt.K + 4) * U32 + unit) * mag
    within(val(out.t), want, err + u * (np.abs(want) + err), f"{fmt} out")
    out.check("out")
    return used


CASES = [(1, 8, 32), (1, 64, 64), (9, 12296, 64), (32, 12328, 160), (2, 72, 96), (3, 16, 288), (16, 264, 160), (17, 136, 544), (31, 6152, 96),
         (5, 6168, 288), (32, 40, 2880), (33, 520, 256), (64, 136, 320), (127, 392, 1056), (129, 264, 512),
         (300, 200, 1312), (513, 392, 800)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,N,K", CASES)
def test_linear_forward(T, N, K, fmt):
    wt = Weight("fwd", N, K, bias=T % 2 == 1)
    used = check(wt, fmt, T, moe4.MOE4_VARIANT_AUTO, BF, BF if N % 16 else F32)
    assert used == (SKINNY if T <= 32 and T * N <= 384 * 1024 or T <= 64 and N <= 2048 else TILED)
    for v in (SKINNY, TILED):
        assert check(wt, fmt, T, v, F32, F32 if T % 3 else None) == v


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,N,K", [(4100, 3080, 160), (2600, 5144, 288), (2600, 5144, 32), (2100, 3080, 1088)])
def test_linear_forward_many_tiles(T, N, K, fmt):
    # enough tiles for the larger shape, ragged on every side
    check(Weight("many", N, K, True), fmt, T, TILED, BF, BF)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,N,K", [(70, 136, 2080), (130, 264, 4160), (97, 8, 8224), (200, 392, 4704), (1, 1032, 16416)])
def test_linear_forward_split_k(T, N, K, fmt):
    wt = Weight("split", N, K, True)
    check(wt, fmt, T, TILED, BF, F32)
    check(wt, fmt, T, TILED, F32, None)


@pytest.mark.parametrize("variant", [SKINNY, TILED])
@pytest.mark.parametrize("fmt", FORMATS)
def test_linear_every_weight_code_and_scale(fmt, variant):
    # row n holds each code twice at scale n; token t picks value t
    codes = (np.arange(32) % 16).astype(np.uint8)
    q = np.tile((codes[0::2] | codes[1::2] << 4)[None, None], (256, 1, 1)).astype(np.uint8)
    s = np.arange(256, dtype=np.uint8)[:, None]
    w = block4.values_mxfp4(q, s)
    lin = moe4.Linear(to_dev(q), to_dev(s), N=256, K=32, variant=variant)
    eye = np.eye(32)
    x, xs = to_dev(bf16_bits_from_f32(eye.astype(np.float32))), None
    if fmt == "mx8":
        x, xs = to_dev((eye * 0x38).astype(np.uint8)), to_dev(np.full((32, 1), 127, np.uint8))
    if fmt == "mx4":
        e = (eye * 2).astype(np.uint8)
        x, xs = to_dev((e[:, 0::2] | e[:, 1::2] << 4).reshape(32, 1, 16)), to_dev(np.full((32, 1), 127, np.uint8))
    out = out_t((32, 256), F32)
    ws = torch.empty(moe4.moe4_linear_workspace_size(lin, 32), dtype=torch.uint8, device="cuda")
    moe4.moe4_linear_forward(lin, x, out.t, x_s=xs, ws=ws)
    got = out.t.double().cpu().numpy()
    assert np.isnan(got[:, 255]).all()
    # scales 253 and 254 hold values past fp32's range, infinities that times 0 may be NaNs
    got, want = got[:, :253], w.T[:, :253]
    small = np.abs(want) < 2.0 ** -126   # not normal: may become zero
    assert np.array_equal(got[~small], want[~small]) and (np.abs(got[small] - want[small]) < 2.0 ** -126).all()


@pytest.mark.parametrize("variant", [SKINNY, TILED])
@pytest.mark.parametrize("fmt", ["mx8", "mx4"])
def test_linear_every_activation_code_and_scale(fmt, variant):
    per = 256 if fmt == "mx8" else 32
    blocks = per // 32
    T = 256 * blocks
    q = (32 * (np.arange(T) % blocks)[:, None] + np.arange(32)).astype(np.uint8)
    s = (np.arange(T) // blocks).astype(np.uint8)[:, None]
    if fmt == "mx4":
        q = q % 16
        q = (q[:, 0::2] | q[:, 1::2] << 4).reshape(T, 1, 16)
        xv = block4.values_mxfp4(q, s)
    else:
        xv = dense.mxfp8_values(q, s)
    e = (np.eye(32) * 2).astype(np.uint8)
    w = (e[:, 0::2] | e[:, 1::2] << 4).reshape(32, 1, 16)
    lin = moe4.Linear(to_dev(w), to_dev(np.full((32, 1), 127, np.uint8)), N=32, K=32, variant=variant)
    out = out_t((T, 32), F32)
    ws = torch.empty(moe4.moe4_linear_workspace_size(lin, T), dtype=torch.uint8, device="cuda")
    moe4.moe4_linear_forward(lin, to_dev(q), out.t, x_s=to_dev(s), ws=ws)
    got = out.t.double().cpu().numpy()
    bad = np.isnan(xv).any(1)
    assert np.isnan(got[bad]).all() and bad[s[:, 0] == 255].all()
    ok = ~bad & (np.abs(xv) < 3.38e38).all(1)   # (an infinity times 0 is a NaN)
    got, want = got[ok], xv[ok]
    small = np.abs(want) < 2.0 ** -126
    assert np.array_equal(got[~small], want[~small]) and (np.abs(got[small] - want[small]) <= 2.0 ** -126).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("variant", [SKINNY, TILED])
def test_linear_non_finite_stay_apart(fmt, variant):
    # tokens, and rows of the weight, next to ends of k inside a tile
    wt = Weight("nan", 96, 96, True)
    T = 20
    lin = wt.lin.with_variant(variant)
    x, xs, _ = tokens(fmt, T, 96)
    clean = torch.empty((T, 96), dtype=BF, device="cuda")
    moe4.moe4_linear_forward(lin, x, clean, x_s=xs, ws=wt.ws(T))
    if fmt == "bf16":
        x[7, 3], x[11, 95] = float("nan"), float("inf")
    else:
        xs[7, 0], xs[11, 2] = 255, 255
    lin.tensors[1][40, 2] = 255
    out = torch.empty_like(clean)
    moe4.moe4_linear_forward(lin, x, out, x_s=xs, ws=wt.ws(T))
    o = val(out)
    t = [i for i in range(T) if i not in (7, 11)]
    n = [i for i in range(96) if i != 40]
    assert torch.equal(out[t][:, n], clean[t][:, n])
    assert np.isnan(o[7]).all() and not np.isfinite(o[11]).any() and np.isnan(o[:, 40]).all()
    dy, _ = draw(rng("nan dy"), (T, 96))
    base, dx = (torch.empty((T, 96), dtype=BF, device="cuda") for _ in range(2))
    lin.tensors[1][40, 2] = 127
    moe4.moe4_linear_backward(lin, dy, base, ws=wt.ws(T, True))
    dy[7, 3] = float("nan")
    lin.tensors[1][40, 2] = 255     # reaches columns 64 .. 95 of every token
    moe4.moe4_linear_backward(lin, dy, dx, ws=wt.ws(T, True))
    t = [i for i in range(T) if i != 7]
    assert torch.equal(dx[t][:, :64], base[t][:, :64])
    assert dx[:, 64:].isnan().all() and dx[7].isnan().all()


def test_linear_in_place_residual():
    wt = Weight("inplace", 264, 160)
    for T in (5, 200):
        x, _, _ = tokens("bf16", T, 160)
        res, _ = draw(rng("r", T), (T, 264))
        out, both = torch.empty_like(res), res.clone()
        moe4.moe4_linear_forward(wt.lin, x, out, residual=res, ws=wt.ws(T))
        moe4.moe4_linear_forward(wt.lin, x, both, residual=both, ws=wt.ws(T))
        assert torch.equal(out, both)
        dy, _ = draw(rng("dy", T), (T, 264))
        add, _ = draw(rng("add", T), (T, 160))
        dx, both = torch.empty_like(add), add.clone()
        moe4.moe4_linear_backward(wt.lin, dy, dx, dx_add=add, ws=wt.ws(T, True))
        moe4.moe4_linear_backward(wt.lin, dy, both, dx_add=both, ws=wt.ws(T, True))
        assert torch.equal(dx, both)


BWD = [(1, 8, 32), (2, 72, 96), (16, 264, 160), (33, 520, 288), (64, 136, 320), (127, 392, 1056), (129, 200, 512),
       (300, 1312, 224), (513, 800, 392 - 8), (70, 2080, 160), (130, 4160, 288), (1, 16392, 64), (4100, 160, 3104),
       (2600, 264, 5152), (2600, 8, 5152)]


@pytest.mark.parametrize("T,N,K", BWD)
def test_linear_backward(T, N, K):
    wt = Weight("bwd", N, K)
    dy, dyv = draw(rng("lin dy", T, N), (T, N))
    for xd, ad, bd in ((BF, F32, F32), (F32, None, BF), (BF, BF, None), (F32, F32, F32)):
        add, av = draw(rng("add", T, K), (T, K), ad) if ad is not None else (None, None)
        dx, db = out_t((T, K), xd), out_t((N,), bd or F32)
        moe4.moe4_linear_backward(wt.lin, dy, dx.t, dx_add=add, db=db.t if bd else None, ws=wt.ws(T, True))
        wx, wb = block4.linear_backward(dyv, wt.w, av)
        mag = np.abs(dyv) @ np.abs(wt.w) + (0 if av is None else np.abs(av))
        err = (N + 4) * U32 * mag
        within(val(dx.t), wx, err + (0 if xd == F32 else ueps(xd)) * (np.abs(wx) + err), "dx")
        dx.check("dx")
        db.check("db")
        if bd:
            err = (T + 4) * U32 * np.abs(dyv).sum(0)
            within(val(db.t), wb, err + (0 if bd == F32 else ueps(bd)) * (np.abs(wb) + err), "db")
        else:
            assert bool((db.raw == 0xA5).all())
    if T < 600:   # db alone
        db = out_t((N,), F32)
        moe4.moe4_linear_backward(wt.lin, dy, db=db.t, ws=wt.ws(T, True))
        within(val(db.t), dyv.sum(0), (T + 4) * U32 * np.abs(dyv).sum(0), "db alone")


def test_linear_backward_every_code_and_scale():
    # token t picks row t, whose scale is t
    codes = (np.arange(32) % 16).astype(np.uint8)
    q = np.tile((codes[0::2] | codes[1::2] << 4)[None, None], (256, 1, 1)).astype(np.uint8)
    s = np.arange(256, dtype=np.uint8)[:, None]
    s[253:] = 127     # (NaN and infinities, which times 0 reach every token)
    w = block4.values_mxfp4(q, s)
    lin = moe4.Linear(to_dev(q), to_dev(s), N=256, K=32)
    dy = to_dev(bf16_bits_from_f32(np.eye(256, dtype=np.float32)))
    dx = out_t((256, 32), F32)
    ws = torch.empty(moe4.moe4_linear_workspace_size(lin, 256, True), dtype=torch.uint8, device="cuda")
    moe4.moe4_linear_backward(lin, dy, dx.t, ws=ws)
    got = dx.t.double().cpu().numpy()
    small = np.abs(w) < 2.0 ** -126
    assert np.array_equal(got[~small], w[~small]) and (np.abs(got[small] - w[small]) < 2.0 ** -126).all()


def test_linear_backward_against_differences():
    # y is linear in x: with integers and h = 1 the quotient is exact but for the fp32 sums
    T, N, K = 40, 136, 96
    wt = Weight("diff", N, K, True)
    r = rng("lin diff")
    x, v, g = (r.integers(-8, 9, s).astype(np.float32) for s in ((T, K), (T, K), (T, N)))

    def y(a):
        out = torch.empty((T, N), device="cuda")
        moe4.moe4_linear_forward(wt.lin, to_dev(bf16_bits_from_f32(a)), out, ws=wt.ws(T))
        return out.double().cpu().numpy()
    dx = torch.empty((T, K), device="cuda")
    moe4.moe4_linear_backward(wt.lin, to_dev(bf16_bits_from_f32(g)), dx, ws=wt.ws(T, True))
    dq = np.sum((y(x + v) - y(x - v)) / 2 * g)
    mag = np.sum((16 * np.abs(wt.w).sum(1) + np.abs(wt.bias)) * np.abs(g))
    assert abs(np.sum(dx.double().cpu().numpy() * v) - dq) <= 2 * (N + K + 8) * U32 * mag


def test_linear_no_tokens():
    wt = Weight("none", 72, 96)
    e = torch.empty((0, 72), dtype=BF, device="cuda")
    moe4.moe4_linear_forward(wt.lin, torch.empty((0, 96), dtype=BF, device="cuda"), e, ws=wt.ws(0))
    for dt in (F32, BF):
        db = out_t((72,), dt)
        moe4.moe4_linear_backward(wt.lin, e, torch.empty((0, 96), dtype=BF, device="cuda"), db=db.t, ws=wt.ws(0, True))
        assert bool((db.t == 0).all())
        db.check("db")


def test_linear_sums_do_not_depend_on_the_run():
    wt = Weight("runs", 264, 4160, True)
    for T in (7, 130):
        x, _, _ = tokens("bf16", T, 4160)
        dy, _ = draw(rng("dy runs", T), (T, 264))
        first = None
        for _ in range(3):
            o, dx, db = (torch.empty(s, device="cuda") for s in ((T, 264), (T, 4160), (264,)))
            moe4.moe4_linear_forward(wt.lin, x, o, ws=wt.ws(T))
            moe4.moe4_linear_backward(wt.lin, dy, dx, db=db, ws=wt.ws(T, True))
            if first is None:
                first = (o, dx, db)
            assert all(torch.equal(a, b) for a, b in zip(first, (o, dx, db)))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,N,K", [(3, 264, 288), (130, 264, 4160), (2600, 5144, 160)])
def test_linear_graph_capture(T, N, K, fmt):
    # captured without an eager call before; replayed with eager work on another workspace between
    wt = Weight("graph", N, K, True)
    x, xs, _ = tokens(fmt, T, K)
    dy, _ = draw(rng("g dy", T, N), (T, N))
    z = [torch.zeros(s, dtype=d, device="cuda") for s, d in (((T, N), BF), ((T, K), BF), ((N,), F32))]
    e = [torch.empty_like(a) for a in z]
    ws, wb, ws2, wb2 = wt.ws(T), wt.ws(T, True), wt.ws(T), wt.ws(T, True)

    def step(o, a, b):
        moe4.moe4_linear_forward(wt.lin, x, o[0], x_s=xs, ws=a)
        moe4.moe4_linear_backward(wt.lin, dy, o[1], db=o[2], ws=b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(z, ws, wb)
    for k in range(3):
        x2, xs2, _ = tokens(fmt, T, K, k + 1)
        x.copy_(x2)
        if xs is not None:
            xs.copy_(xs2)
        dy.copy_(draw(rng("g dy", T, N, k), (T, N))[0])
        for a in z:
            a.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        step(e, ws2, wb2)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(z, e))


def test_linear_two_at_once():
    # the same weight on two streams, each with a workspace of its own
    wt = Weight("two", 264, 4160)
    T = 100
    xa, _, _ = tokens("bf16", T, 4160, 1)
    xb, _, _ = tokens("bf16", T, 4160, 2)
    want = []
    for x in (xa, xb):
        o = torch.empty((T, 264), dtype=BF, device="cuda")
        moe4.moe4_linear_forward(wt.lin, x, o, ws=wt.ws(T))
        want.append(o)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    oa, ob = torch.empty_like(want[0]), torch.empty_like(want[0])
    wa, wb = wt.ws(T), wt.ws(T)
    for s in (sa, sb):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        moe4.moe4_linear_forward(wt.lin, xa, oa, ws=wa, stream=sa)
        with torch.cuda.stream(sb):
            moe4.moe4_linear_forward(wt.lin, xb, ob, ws=wb)
    for s in (sa, sb):
        torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(oa, want[0]) and torch.equal(ob, want[1])


def test_linear_offsets_past_32_bits():
    # tensors of more than 2^32 bytes: the last rows are those of a call on them alone
    T, tail = 1_060_000, 300
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((T, 2048), generator=gen, device="cuda", dtype=BF)
    wt = Weight("huge in", 16, 2048)
    out, o2 = torch.empty((T, 16), device="cuda"), torch.empty((tail, 16), device="cuda")
    moe4.moe4_linear_forward(wt.lin, x, out, ws=wt.ws(T))
    moe4.moe4_linear_forward(wt.lin, x[-tail:].clone(), o2, ws=wt.ws(tail))
    # (the tail's call is cut along k: each sum is off by its own order)
    mag = x[-tail:].double().abs() @ torch.from_numpy(np.abs(wt.w).T.copy()).cuda()
    assert bool(((out[-tail:] - o2).double().abs() <= 2 * (2048 + 4) * U32 * mag).all())
    back = Weight("huge out", 2048, 32)
    dx, d2 = torch.empty((T, 32), device="cuda"), torch.empty((tail, 32), device="cuda")
    moe4.moe4_linear_backward(back.lin, x, dx, ws=back.ws(T, True))
    moe4.moe4_linear_backward(back.lin, x[-tail:].clone(), d2, ws=back.ws(tail, True))
    mag = x[-tail:].double().abs() @ torch.from_numpy(np.abs(back.w)).cuda()
    assert bool(((dx[-tail:] - d2).double().abs() <= 2 * (2048 + 4) * U32 * mag).all())
    dy = x[:, :16].contiguous()
    del out, dx
    y = torch.empty_like(x)
    moe4.moe4_linear_backward(wt.lin, dy, y, ws=wt.ws(T, True))
    e = torch.empty((tail, 2048), dtype=BF, device="cuda")
    moe4.moe4_linear_backward(wt.lin, dy[-tail:].clone(), e, ws=wt.ws(tail, True))
    assert torch.equal(y[-tail:], e)


def test_linear_binding_refusals():
    wt = Weight("bind", 72, 96)
    x, _, _ = tokens("bf16", 4, 96)
    out = torch.empty((4, 72), dtype=BF, device="cuda")
    ws = wt.ws(4)
    E = (moe4.Moe4Error, TypeError, ValueError)
    q, s = wt.lin.tensors[:2]
    for bad in (dict(x=x[:, :64]), dict(x=x.float()), dict(out=out[:3]), dict(residual=out.half()), dict(x_s=s),
                dict(x=x.cpu()), dict(out=out.t().contiguous().t())):
        a = dict(x=x, out=out, ws=ws)
        a.update(bad)
        with pytest.raises(E):
            moe4.moe4_linear_forward(wt.lin, **a)
    with pytest.raises(E):
        moe4.moe4_linear_forward(wt.lin, to_dev(np.zeros((4, 3, 16), np.uint8)), out, ws=ws)   # codes without scales
    with pytest.raises(E):
        moe4.Linear(q, s[:-1].clone(), N=72, K=96)
    with pytest.raises(E):
        moe4.moe4_linear_backward(wt.lin, out, dx_add=x, ws=wt.ws(4, True))
    with pytest.raises(E):
        moe4.moe4_linear_workspace_size(wt.lin, -1)
