"""Refusals of the operators of a block held in 4 bits: every bad argument is named synchronously,
before anything is enqueued, so no call here reaches a device. The same file runs against the
library's ASan build (test_dense_abi_asan.py's way, in test_block4_abi_asan.py)."""
import ctypes

import pytest

moe4 = pytest.importorskip("bit_mixture_experts_amd.moe4")
lib = moe4._lib

P = 0x10000          # 256-byte aligned, never dereferenced: validation fails first
MIS = 0x10004        # 4-byte aligned only
BF, F32 = moe4.MOE4_DTYPE_BF16, moe4.MOE4_DTYPE_F32
OK, EINVAL, EUNSUP, ESHAPE = 0, moe4.MOE4_EINVAL, moe4.MOE4_EUNSUPPORTED, moe4.MOE4_ESHAPE
EALIGN, EWS = moe4.MOE4_EALIGN, moe4.MOE4_EWORKSPACE
X8, X4 = moe4.MOE4_X_MXFP8, moe4.MOE4_X_MXFP4


def refused(rc, code, msg):
    assert rc == code and msg in moe4.moe4_last_error(), (rc, moe4.moe4_last_error())


# ------------------------------------------------------------------- MXFP4

def _q4(**kw):
    a = dict(x=P, xd=BF, R=4, K=64, q=P, s=P, v=None)
    a.update(kw)
    return lib.moe4_quantize_mxfp4(*a.values(), None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(xd=0), EINVAL, "x_dtype unset"), (dict(xd=7), EINVAL, "x_dtype unknown"),
    (dict(R=-1), ESHAPE, "negative"), (dict(K=33), ESHAPE, "K = 33"), (dict(K=-32), ESHAPE, "K = -32"),
    (dict(R=1 << 40, K=64), ESHAPE, "2^40"), (dict(x=None), EINVAL, "x is NULL"),
    (dict(q=None), EINVAL, "blocks is NULL"), (dict(s=None), EINVAL, "scales is NULL"),
    (dict(x=MIS), EALIGN, "x is not"), (dict(q=MIS), EALIGN, "blocks is not"),
    (dict(v=MIS), EALIGN, "values is not"),
])
def test_quantize_refusals(kw, code, msg):
    refused(_q4(**kw), code, msg)


def test_quantize_of_nothing():
    assert _q4(R=0, x=None, q=None, s=None) == OK and _q4(K=0, x=None, q=None, s=None) == OK


# -------------------------------------------------------------------- join

def _join(**kw):
    a = dict(b=P, bd=BF, res=P, sd=BF, rs=1.0, bs=1.0, gate=None, wo=P, od=BF, wi=P, id=BF, T=4, H=64,
             eps=1e-6, sum=P, ro=None, ri=None, out=P, q=None, qs=None, qf=0)
    a.update(kw)
    return lib.moe4_join_norm(*a.values(), None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(H=60), ESHAPE, "H = 60"), (dict(H=16392), ESHAPE, "16384"), (dict(T=-1), ESHAPE, "negative"),
    (dict(bd=0), EINVAL, "b_dtype unset"), (dict(sd=5), EINVAL, "s_dtype unknown"),
    (dict(od=0), EINVAL, "post_dtype unset"), (dict(id=0), EINVAL, "pre_dtype unset"),
    (dict(eps=-1.0), EINVAL, "eps"), (dict(eps=float("nan")), EINVAL, "eps"),
    (dict(q=P), EINVAL, "together"), (dict(q=P, qs=P), EINVAL, "q_format unset"),
    (dict(q=P, qs=P, qf=1), EINVAL, "neither"), (dict(q=P, qs=P, qf=X4, H=72), ESHAPE, "multiple of 32"),
    (dict(b=None), EINVAL, "b is NULL"), (dict(wi=None), EINVAL, "out given without w_pre"),
    (dict(wi=None, out=None, q=P, qs=P, qf=X8), EINVAL, "out_q given without w_pre"),
    (dict(wi=None, out=None, ri=P), EINVAL, "rstd_pre given without w_pre"),
    (dict(wo=None, ro=P), EINVAL, "rstd_post given"), (dict(sum=None, out=None), EINVAL, "all NULL"),
    (dict(out=None), EINVAL, "w_pre given"), (dict(b=MIS), EALIGN, "b is not"),
    (dict(res=MIS), EALIGN, "residual is not"), (dict(gate=P + 2), EALIGN, "gate is not"),
    (dict(wo=MIS), EALIGN, "w_post is not"), (dict(wi=MIS), EALIGN, "w_pre is not"),
    (dict(sum=MIS), EALIGN, "sum_out is not"), (dict(ro=P + 2), EALIGN, "rstd_post is not"),
    (dict(ri=P + 2), EALIGN, "rstd_pre is not"), (dict(out=MIS), EALIGN, "out is not"),
    (dict(q=MIS, qs=P, qf=X8), EALIGN, "out_q is not"),
])
def test_join_refusals(kw, code, msg):
    refused(_join(**kw), code, msg)


def _join_bwd(**kw):
    a = dict(dy=P, yd=BF, s=P, sd=BF, b=P, bd=BF, ds=P, rs=1.0, bs=1.0, gate=None, wo=P, od=BF, wi=P,
             id=BF, ro=P, ri=P, T=4, H=64, db=P, dres=P + 4096, dg=None, dwo=P, dwi=P, ws=P, n=1 << 22)
    a.update(kw)
    return lib.moe4_join_norm_backward(*a.values(), None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(H=12), ESHAPE, "H = 12"), (dict(T=-2), ESHAPE, "negative"), (dict(yd=0), EINVAL, "dy_dtype unset"),
    (dict(sd=0), EINVAL, "s_dtype unset"), (dict(bd=9), EINVAL, "b_dtype unknown"),
    (dict(od=0), EINVAL, "post_dtype unset"), (dict(id=0), EINVAL, "pre_dtype unset"),
    (dict(wi=None), EINVAL, "dy given without w_pre"), (dict(wi=None, dy=None), EINVAL, "s given without"),
    (dict(wi=None, dy=None, s=None), EINVAL, "rstd_pre given"),
    (dict(wi=None, dy=None, s=None, ri=None), EINVAL, "dw_pre given"),
    (dict(wi=None, dy=None, s=None, ri=None, dwi=None, ds=None), EINVAL, "ds is NULL"),
    (dict(wo=None), EINVAL, "rstd_post given"), (dict(wo=None, ro=None), EINVAL, "dw_post given"),
    (dict(dy=None), EINVAL, "dy is NULL"), (dict(s=None), EINVAL, "s is NULL"),
    (dict(ri=None), EINVAL, "rstd_pre is NULL"), (dict(ro=None), EINVAL, "rstd_post is NULL"),
    (dict(b=None), EINVAL, "b is NULL"), (dict(db=None), EINVAL, "db is NULL"),
    (dict(dres=P), EINVAL, "same memory"), (dict(dy=MIS), EALIGN, "dy is not"),
    (dict(s=MIS), EALIGN, "s is not"), (dict(b=MIS), EALIGN, "b is not"), (dict(ds=MIS), EALIGN, "ds is not"),
    (dict(db=MIS), EALIGN, "db is not"), (dict(dres=MIS), EALIGN, "dres is not"),
    (dict(dg=P + 1), EALIGN, "dgate is not"), (dict(dwo=MIS), EALIGN, "dw_post is not"),
    (dict(dwi=MIS), EALIGN, "dw_pre is not"), (dict(ws=None), EWS, "needed"), (dict(n=16), EWS, "16 bytes"),
    (dict(ws=P + 16), EALIGN, "256-byte"),
])
def test_join_backward_refusals(kw, code, msg):
    refused(_join_bwd(**kw), code, msg)


def test_join_of_no_rows_and_workspace():
    assert _join(T=0, b=None, res=None, sum=None, out=None) == OK
    assert _join_bwd(T=0, dy=None, s=None, b=None, ds=None, db=None, dres=None, dwo=None, dwi=None, ws=None,
                     n=0, ro=None, ri=None) == OK
    assert lib.moe4_join_norm_workspace_size(4, 60) == 0 and lib.moe4_join_norm_workspace_size(-1, 64) == 0
    for H in (64, 1024, 2880, 16384):   # never falls as the rows grow
        sizes = [lib.moe4_join_norm_workspace_size(T, H) for T in (0, 1, 7, 500, 2047, 2048, 2049, 8192, 1 << 30)]
        assert sizes == sorted(sizes) and sizes[0] >= 256 and sizes[-1] <= 2048 * H * 8


# ------------------------------------------------------------------- layer

def _ex(**kw):
    a = dict(format=moe4.MOE4_FMT_NF4, E=8, H=128, I=64, gu_layout=1, act=1, act_alpha=1.702, act_limit=7.0,
             gu_q=P, gu_s=P, dn_q=P, dn_s=P)
    a.update(kw)
    return moe4.Moe4Experts(**a)


def _layer(ex=None, **kw):
    a = dict(x=P, lg=P, T=4, k=2, rn=1, res=None, rd=0, out=P, od=BF, idx=None, w=None, ws=P, n=1 << 24)
    a.update(kw)
    return lib.moe4_layer_decode(ctypes.byref(ex if ex is not None else _ex()), *a.values(), None)


@pytest.mark.parametrize("ex,kw,code,msg", [
    (dict(format=0), {}, EINVAL, "format unset"), (dict(act=0), {}, EINVAL, "act unset"),
    (dict(H=100), {}, ESHAPE, "H = 100"), (dict(gu_q=None), {}, EINVAL, "gu_q is NULL"),
    (dict(lora_A=P, lora_B=P, lora_r=4, lora_scale=1.0), {}, EUNSUP, "adapters"),
    (dict(variant=moe4.MOE4_VARIANT_TILED), {}, EUNSUP, "TILED"),
    (dict(format=moe4.MOE4_FMT_NF4_DQ, gu_s2=P, dn_s2=P, gu_soff=P, dn_soff=P, dq_book=P, H=16448), {}, EUNSUP,
     "16384"),
    ({}, dict(T=33), ESHAPE, "T = 33"), ({}, dict(T=-1), ESHAPE, "T = -1"), ({}, dict(k=0), ESHAPE, "k = 0"),
    ({}, dict(k=9), ESHAPE, "k = 9"), (dict(E=32), dict(T=32, k=17), ESHAPE, "512 slots"),
    ({}, dict(od=0), EINVAL, "out_dtype unset"), ({}, dict(res=P), EINVAL, "res_dtype unset"),
    ({}, dict(x=None), EINVAL, "x is NULL"), ({}, dict(lg=None), EINVAL, "logits is NULL"),
    ({}, dict(out=None), EINVAL, "out is NULL"), ({}, dict(x=MIS), EALIGN, "x is not"),
    ({}, dict(lg=P + 2), EALIGN, "logits is not"), ({}, dict(res=MIS, rd=BF), EALIGN, "residual is not"),
    ({}, dict(out=MIS), EALIGN, "out is not"), ({}, dict(idx=P + 1), EALIGN, "topk_idx is not"),
    ({}, dict(w=P + 2), EALIGN, "topk_w is not"), ({}, dict(ws=None), EWS, "needed"),
    ({}, dict(n=64), EWS, "64 bytes given"), ({}, dict(ws=P + 16), EALIGN, "256-byte"),
])
def test_layer_refusals(ex, kw, code, msg):
    refused(_layer(_ex(**ex), **kw), code, msg)


def test_layer_of_no_tokens_and_workspace():
    assert _layer(T=0, x=None, lg=None, out=None, ws=None, n=0) == OK
    e = _ex()
    size = lambda T, k: lib.moe4_layer_decode_workspace_size(ctypes.byref(e), T, k)   # noqa: E731
    assert size(33, 2) == 0 and size(4, 9) == 0 and size(0, 2) >= 256
    sizes = [size(T, 8) for T in range(33)]
    assert sizes == sorted(sizes)


# ------------------------------------------------------------------ linear

def _lin(**kw):
    d = dict(N=64, K=64, variant=moe4.MOE4_VARIANT_AUTO, w_q=P, w_s=P, bias=None)
    d.update(kw)
    return ctypes.byref(moe4.Moe4Linear(**d))


def _lin_fwd(lin=None, **kw):
    a = dict(x=P, fmt=moe4.MOE4_X_BF16, xs=None, T=4, res=None, rd=0, out=P, od=BF, ws=P, n=1 << 30)
    a.update(kw)
    return lib.moe4_linear_forward(_lin(**(lin or {})), *a.values(), None)


def _lin_bwd(lin=None, **kw):
    a = dict(dy=P, T=4, add=None, ad=0, dx=P, xd=BF, db=P, bd=F32, ws=P, n=1 << 30)
    a.update(kw)
    return lib.moe4_linear_backward(_lin(**(lin or {})), *a.values(), None)


LINEAR = [
    (dict(N=0), ESHAPE, "N = 0"), (dict(N=12), ESHAPE, "N = 12"), (dict(K=48), ESHAPE, "K = 48"),
    (dict(K=-32), ESHAPE, "K = -32"), (dict(N=1 << 16, K=1 << 16), ESHAPE, "under 2 GiB"),
    (dict(N=1 << 21, K=32), ESHAPE, "256 rows"), (dict(variant=9), EINVAL, "variant unknown"),
    (dict(w_q=None), EINVAL, "w_q is NULL"), (dict(w_s=None), EINVAL, "w_s is NULL"),
    (dict(w_q=MIS), EALIGN, "w_q is not"), (dict(w_s=P + 2), EALIGN, "w_s is not"),
    (dict(bias=MIS), EALIGN, "bias is not"),
]


@pytest.mark.parametrize("lin,code,msg", LINEAR)
def test_linear_descriptor_refusals(lin, code, msg):
    refused(_lin_fwd(lin), code, msg)
    refused(_lin_bwd(lin), code, msg)
    assert lib.moe4_linear_workspace_size(_lin(**lin), 4, 0) == 0
    assert lib.moe4_linear_workspace_size(_lin(**lin), 4, 1) == 0


def test_linear_without_descriptor():
    refused(lib.moe4_linear_forward(None, P, 1, None, 4, None, 0, P, BF, P, 1 << 30, None), EINVAL, "moe4_linear is NULL")
    refused(lib.moe4_linear_backward(None, P, 4, None, 0, P, BF, P, F32, P, 1 << 30, None), EINVAL, "moe4_linear is NULL")


@pytest.mark.parametrize("lin,kw,code,msg", [
    ({}, dict(fmt=0), EINVAL, "x_format unset"), ({}, dict(fmt=4), EINVAL, "x_format unknown"),
    ({}, dict(od=0), EINVAL, "out_dtype unset"), ({}, dict(res=P, rd=3), EINVAL, "res_dtype unknown"),
    ({}, dict(xs=P), EINVAL, "x_s given"), ({}, dict(fmt=X8), EINVAL, "x_s is NULL"),
    ({}, dict(fmt=X4), EINVAL, "x_s is NULL"), ({}, dict(T=-1), ESHAPE, "negative"),
    ({}, dict(x=None), EINVAL, "x is NULL"), ({}, dict(out=None), EINVAL, "out is NULL"),
    ({}, dict(x=MIS), EALIGN, "x is not"), ({}, dict(fmt=X8, xs=P + 2), EALIGN, "x_s is not"),
    ({}, dict(res=MIS, rd=BF), EALIGN, "residual is not"), ({}, dict(out=MIS), EALIGN, "out is not"),
    (dict(K=4096), dict(ws=None), EWS, "workspace of 0 bytes"), (dict(K=4096), dict(T=64, n=256), EWS, "workspace"),
    (dict(K=4096), dict(ws=MIS), EALIGN, "256"), (dict(variant=moe4.MOE4_VARIANT_SKINNY), dict(T=(1 << 20) + 1), ESHAPE, "2^20"),
    (dict(K=1 << 20, N=8), dict(T=1 << 17), ESHAPE, "scales"),
    (dict(N=1 << 18, K=32), dict(T=1 << 18), ESHAPE, "scales"), (dict(N=8, K=32), dict(T=1 << 30), ESHAPE, "launch"),
])
def test_linear_refusals(lin, kw, code, msg):
    refused(_lin_fwd(lin, **kw), code, msg)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(xd=0), EINVAL, "dx_dtype unset"), (dict(dx=None, add=P, ad=BF), EINVAL, "dx_add given without dx"),
    (dict(add=P, ad=5), EINVAL, "add_dtype unknown"), (dict(bd=0), EINVAL, "db_dtype unset"),
    (dict(dy=None), EINVAL, "dy is NULL"), (dict(dy=MIS), EALIGN, "dy is not"),
    (dict(add=MIS, ad=BF), EALIGN, "dx_add is not"), (dict(dx=MIS), EALIGN, "dx is not"),
    (dict(db=MIS), EALIGN, "db is not"), (dict(n=256), EWS, "workspace"), (dict(T=-3), ESHAPE, "negative"),
])
def test_linear_backward_refusals(kw, code, msg):
    refused(_lin_bwd(**kw), code, msg)


def test_linear_of_nothing_and_workspace():
    assert _lin_fwd(T=0, x=None, out=None, ws=None, n=0) == OK
    assert _lin_bwd(T=0, dy=None, dx=None, db=None, ws=None, n=0) == OK
    assert _lin_bwd(dy=None, dx=None, db=None, ws=None, n=0) == OK
    for lin in (dict(), dict(N=264, K=4160), dict(N=8, K=16384), dict(N=16384, K=32), dict(N=4096, K=4096)):
        for back in (0, 1):   # never less than for fewer tokens
            last = 0
            for T in (0, 1, 16, 17, 33, 64, 129, 500, 1000, 4096, 70000):
                n = lib.moe4_linear_workspace_size(_lin(**lin), T, back)
                assert n >= max(last, 256)
                last = n
    assert lib.moe4_linear_workspace_size(_lin(), -1, 0) == 0
