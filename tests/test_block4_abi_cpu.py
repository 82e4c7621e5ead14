"""Refusals of the operators of a block held in 4 bits: every bad argument is named synchronously,
before anything is enqueued, so no call here reaches a device. The same file runs against the
library's ASan build (test_dense_abi_asan.py's way, in test_block4_abi_asan.py)."""
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
