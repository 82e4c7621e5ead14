"""Refusals of the dense operators (norm, MXFP8, feed-forward block, gradient clipping): every
bad argument is named synchronously, before anything is enqueued, so no call here reaches a
device. The same file runs against the library's ASan build (test_dense_abi_asan.py)."""
import ctypes

import pytest
import torch

moe4 = pytest.importorskip("bit_mixture_experts_amd.moe4")
lib = moe4._lib

P = 0x10000          # 256-byte aligned, never dereferenced: validation fails first
MIS = 0x10004        # 4-byte aligned only
BF, F32 = moe4.MOE4_DTYPE_BF16, moe4.MOE4_DTYPE_F32
OK, EINVAL, EUNSUP, ESHAPE = 0, moe4.MOE4_EINVAL, moe4.MOE4_EUNSUPPORTED, moe4.MOE4_ESHAPE
EALIGN, EWS = moe4.MOE4_EALIGN, moe4.MOE4_EWORKSPACE


def _norm(**kw):
    a = dict(x=P, xd=BF, res=P, rd=BF, sum=P, w=P, wd=BF, T=4, H=64, eps=1e-6, out=P, q=None, qs=None,
             rstd=None)
    a.update(kw)
    return lib.moe4_add_rmsnorm(*a.values(), None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(H=60), ESHAPE, "H = 60"), (dict(H=0), ESHAPE, "H = 0"), (dict(H=16392), ESHAPE, "16384"),
    (dict(T=-1), ESHAPE, "negative"), (dict(xd=0), EINVAL, "x_dtype unset"),
    (dict(wd=3), EINVAL, "w_dtype unknown"), (dict(rd=0), EINVAL, "res_dtype unset"),
    (dict(eps=-1.0), EINVAL, "eps"), (dict(eps=float("nan")), EINVAL, "eps"),
    (dict(res=None), EINVAL, "without a residual"), (dict(q=P), EINVAL, "together"),
    (dict(q=P, qs=P, H=72), ESHAPE, "multiple of 32"), (dict(out=None), EINVAL, "both NULL"),
    (dict(x=None), EINVAL, "x is NULL"), (dict(w=None), EINVAL, "weight is NULL"),
    (dict(x=MIS), EALIGN, "x is not"), (dict(res=MIS), EALIGN, "residual is not"),
    (dict(sum=MIS), EALIGN, "sum_out is not"), (dict(w=MIS), EALIGN, "weight is not"),
    (dict(out=MIS), EALIGN, "out is not"), (dict(q=MIS, qs=P), EALIGN, "out_q is not"),
    (dict(rstd=P + 2), EALIGN, "rstd is not"),
])
def test_norm_refusals(kw, code, msg):
    assert _norm(**kw) == code
    assert msg in moe4.moe4_last_error()


def test_norm_of_no_rows():
    assert _norm(T=0, x=None, res=None, sum=None, w=None, out=None) == OK
    assert moe4.moe4_last_error() == ""


def _norm_bwd(**kw):
    a = dict(dy=P, yd=BF, s=P, sd=BF, w=P, wd=BF, rstd=P, dres=P, T=4, H=64, dx=P, dd=BF, dw=P, ws=P,
             n=1 << 20)
    a.update(kw)
    return lib.moe4_add_rmsnorm_backward(*a.values(), None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(H=12), ESHAPE, "H = 12"), (dict(T=-2), ESHAPE, "negative"),
    (dict(yd=0), EINVAL, "dy_dtype unset"), (dict(sd=9), EINVAL, "s_dtype unknown"),
    (dict(dd=0), EINVAL, "dx_dtype unset"), (dict(wd=0), EINVAL, "w_dtype unset"),
    (dict(dy=None), EINVAL, "dy is NULL"), (dict(s=None), EINVAL, "s is NULL"),
    (dict(rstd=None), EINVAL, "rstd is NULL"), (dict(dx=None), EINVAL, "dx is NULL"),
    (dict(w=None), EINVAL, "weight is NULL"),
    (dict(dy=MIS), EALIGN, "dy is not"), (dict(s=MIS), EALIGN, "s is not"),
    (dict(dres=MIS), EALIGN, "dres is not"), (dict(dx=MIS), EALIGN, "dx is not"),
    (dict(dw=MIS), EALIGN, "dweight is not"), (dict(ws=None), EWS, "needed"),
    (dict(n=16), EWS, "16 bytes given"), (dict(ws=P + 16), EALIGN, "256-byte"),
])
def test_norm_backward_refusals(kw, code, msg):
    assert _norm_bwd(**kw) == code
    assert msg in moe4.moe4_last_error()


def test_norm_workspace():
    assert lib.moe4_add_rmsnorm_workspace_size(4, 60) == 0
    assert lib.moe4_add_rmsnorm_workspace_size(-1, 64) == 0
    assert lib.moe4_add_rmsnorm_workspace_size(0, 64) >= 256
    big = lib.moe4_add_rmsnorm_workspace_size(1 << 30, 16384)
    assert 0 < big <= 2048 * 16384 * 4   # a bounded number of rows of partial sums
    with pytest.raises(moe4.Moe4Error):
        moe4.moe4_add_rmsnorm_workspace_size(4, 60)


def test_quantize_mxfp8_refusals():
    q = lib.moe4_quantize_mxfp8
    assert q(P, 0, 4, 64, P, P, None) == EINVAL and "x_dtype unset" in moe4.moe4_last_error()
    assert q(P, BF, -1, 64, P, P, None) == ESHAPE
    assert q(P, BF, 4, 48, P, P, None) == ESHAPE and "multiple of 32" in moe4.moe4_last_error()
    assert q(P, BF, 1 << 40, 64, P, P, None) == ESHAPE
    assert q(None, BF, 4, 64, P, P, None) == EINVAL
    assert q(P, BF, 4, 64, None, P, None) == EINVAL
    assert q(P, BF, 4, 64, P, None, None) == EINVAL
    assert q(MIS, BF, 4, 64, P, P, None) == EALIGN
    assert q(P, BF, 4, 64, MIS, P, None) == EALIGN
    assert q(None, F32, 0, 64, None, None, None) == OK
    assert q(None, F32, 4, 0, None, None, None) == OK


def _desc(**kw):
    d = moe4.Moe4Ffn(format=moe4.MOE4_FFN_BF16, H=64, I=96, gu_layout=moe4.MOE4_GU_HALVES,
                     act=moe4.MOE4_ACT_SWIGLU, act_alpha=1.702, act_limit=7.0, variant=0, w_gu=P,
                     w_dn=P)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _fwd(d, **kw):
    a = dict(x=P, xs=None, T=4, res=P, rd=BF, out=P, od=BF, gu=None, ws=P, n=1 << 30)
    a.update(kw)
    return lib.moe4_ffn_forward(ctypes.byref(d), *a.values(), None)


MX = dict(format=moe4.MOE4_FFN_MXFP8, gu_s=P, dn_s=P)


@pytest.mark.parametrize("field,code,msg", [
    (dict(format=0), EINVAL, "format unset"), (dict(format=5), EINVAL, "format unknown"),
    (dict(gu_layout=0), EINVAL, "gu_layout unset"), (dict(act=0), EINVAL, "act unset"),
    (dict(variant=9), EINVAL, "variant unknown"), (dict(H=60), ESHAPE, "H = 60"),
    (dict(H=0), ESHAPE, "H = 0"), (dict(I=-8), ESHAPE, "I = -8"), (dict(I=4), ESHAPE, "multiple of 8"),
    (dict(H=1 << 15, I=1 << 15), ESHAPE, "under 2 GiB"), (dict(H=8, I=1 << 22), ESHAPE, "256 rows"),
    (dict(w_gu=None), EINVAL, "w_gu is NULL"), (dict(w_dn=None), EINVAL, "w_dn is NULL"),
    (dict(w_gu=MIS), EALIGN, "w_gu is not"), (dict(w_dn=MIS), EALIGN, "w_dn is not"),
    (dict(gu_s=P), EINVAL, "scales given"), (dict(gu_bias=P + 2), EALIGN, "gu_bias is not"),
    (dict(dn_bias=P + 8), EALIGN, "dn_bias is not"),
    (dict(act=moe4.MOE4_ACT_SWIGLU_CLAMPED, act_limit=0.0), EINVAL, "act_limit"),
    (dict(act=moe4.MOE4_ACT_SWIGLU_CLAMPED, act_alpha=float("nan")), EINVAL, "act_alpha"),
    ({**MX, "H": 72}, ESHAPE, "multiple of 32"), ({**MX, "I": 72}, ESHAPE, "multiple of 32"),
    ({**MX, "dn_s": None}, EINVAL, "dn_s is NULL"), ({**MX, "gu_s": P + 2}, EALIGN, "gu_s is not"),
])
def test_ffn_descriptor_refusals(field, code, msg):
    d = _desc(**field)
    assert _fwd(d, xs=P if field.get("format") == moe4.MOE4_FFN_MXFP8 else None) == code
    assert msg in moe4.moe4_last_error()
    assert moe4.moe4_last_variant() == 0
    assert lib.moe4_ffn_workspace_size(ctypes.byref(d), 4, 0) == 0


@pytest.mark.parametrize("kw,code,msg", [
    (dict(T=-1), ESHAPE, "negative"), (dict(od=0), EINVAL, "out_dtype unset"),
    (dict(rd=0), EINVAL, "res_dtype unset"), (dict(xs=P), EINVAL, "x_s given"),
    (dict(x=None), EINVAL, "x is NULL"), (dict(out=None), EINVAL, "out is NULL"),
    (dict(x=MIS), EALIGN, "x is not"), (dict(res=MIS), EALIGN, "residual is not"),
    (dict(out=MIS), EALIGN, "out is not"), (dict(gu=MIS), EALIGN, "save_gu is not"),
    (dict(ws=None), EWS, "needed"), (dict(n=255), EWS, "255 bytes"), (dict(ws=P + 8), EALIGN, "256-byte"),
])
def test_ffn_forward_refusals(kw, code, msg):
    assert _fwd(_desc(), **kw) == code
    assert msg in moe4.moe4_last_error()


def test_ffn_forward_other_refusals():
    assert lib.moe4_ffn_forward(None, P, None, 4, None, 0, P, BF, None, P, 1 << 30, None) == EINVAL
    assert _fwd(_desc(**MX)) == EINVAL and "x_s is NULL" in moe4.moe4_last_error()
    assert _fwd(_desc(**MX), xs=P + 1) == EALIGN
    assert _fwd(_desc(variant=moe4.MOE4_VARIANT_SKINNY), T=(1 << 20) + 1) == ESHAPE
    assert "skinny" in moe4.moe4_last_error()
    assert _fwd(_desc(H=1 << 20, I=64), T=1 << 30) == ESHAPE
    assert _fwd(_desc(), T=0, x=None, out=None, ws=None, n=0) == OK


def test_ffn_workspace():
    d = _desc()
    ws = lib.moe4_ffn_workspace_size
    assert ws(ctypes.byref(d), 4, 0) == 4 * 96 * 2
    assert ws(ctypes.byref(_desc(**MX)), 5, 0) == 512 + 256
    assert ws(ctypes.byref(d), 4, 1) >= 4 * 2 * 96 * 2 + 4 * 96 * 2
    assert ws(ctypes.byref(d), 0, 0) >= 256 and ws(ctypes.byref(d), -1, 0) == 0
    assert ws(None, 4, 0) == 0


def _bwd(d, **kw):
    a = dict(x=P, T=4, gu=P, dy=P, add=P, ad=BF, dx=P, dd=BF, wg=P, wdn=P, bg=P, bd=P, wd=BF, ws=P,
             n=1 << 30)
    a.update(kw)
    return lib.moe4_ffn_backward(ctypes.byref(d), *a.values(), None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(T=-1), ESHAPE, "negative"), (dict(dd=0), EINVAL, "dx_dtype unset"),
    (dict(ad=0), EINVAL, "add_dtype unset"), (dict(dx=None), EINVAL, "without dx"),
    (dict(wd=0), EINVAL, "dw_dtype unset"), (dict(dy=None), EINVAL, "dy is NULL"),
    (dict(gu=None), EINVAL, "save_gu is NULL"), (dict(x=None), EINVAL, "x is NULL"),
    (dict(x=MIS), EALIGN, "x is not"), (dict(gu=MIS), EALIGN, "save_gu is not"),
    (dict(dy=MIS), EALIGN, "dy is not"), (dict(add=MIS), EALIGN, "dx_add is not"),
    (dict(dx=MIS), EALIGN, "dx is not"), (dict(wg=MIS), EALIGN, "dw_gu is not"),
    (dict(wdn=MIS), EALIGN, "dw_dn is not"), (dict(bg=MIS), EALIGN, "db_gu is not"),
    (dict(bd=MIS), EALIGN, "db_dn is not"), (dict(ws=None), EWS, "needed"), (dict(n=64), EWS, "64 bytes"),
])
def test_ffn_backward_refusals(kw, code, msg):
    assert _bwd(_desc(), **kw) == code
    assert msg in moe4.moe4_last_error()


def test_ffn_backward_other_refusals():
    assert _bwd(_desc(**MX)) == EUNSUP and "bf16 blocks only" in moe4.moe4_last_error()
    # nothing wanted, nothing read
    assert _bwd(_desc(), x=None, gu=None, dy=None, add=None, dx=None, wg=None, wdn=None, bg=None,
                bd=None, ws=None, n=0) == OK
    assert _bwd(_desc(), T=0, x=None, gu=None, dy=None, add=None, dx=None, wg=None, wdn=None, bg=None,
                bd=None, ws=None, n=0) == OK


def _list(ptrs, numel, dtype, outs=None):
    n = len(ptrs)
    arr = (ctypes.c_void_p * n)(*ptrs)
    o = None if outs is None else (ctypes.c_void_p * n)(*outs)
    return arr, o, (ctypes.c_int64 * n)(*numel), (ctypes.c_int32 * n)(*dtype), n


def test_grad_refusals():
    def norm(*a, out=P, ws=P, nb=1 << 20):
        arr, _, nu, dt, n = _list(*a)
        return lib.moe4_grad_norm(arr, nu, dt, n, out, ws, nb, None)

    def clip(*a, mx=1.0, ni=None, no=P, ws=P, nb=1 << 20):
        arr, o, nu, dt, n = _list(*a)
        return lib.moe4_clip_grads(arr, o, nu, dt, n, mx, ni, no, ws, nb, None)

    assert norm([P], [-1], [BF]) == ESHAPE and "numel[0]" in moe4.moe4_last_error()
    assert norm([P], [(1 << 36) + 1], [BF]) == ESHAPE
    assert norm([P, P], [4, 4], [BF, 0]) == EINVAL and "dtype[1]" in moe4.moe4_last_error()
    assert norm([P, None], [4, 4], [BF, BF]) == EINVAL and "grads[1] is NULL" in moe4.moe4_last_error()
    assert norm([MIS], [4], [BF]) == EALIGN
    assert norm([P], [4], [BF], out=None) == EINVAL
    assert norm([P], [4], [BF], ws=None) == EWS and norm([P], [4], [BF], nb=8) == EWS
    assert lib.moe4_grad_norm(None, None, None, -1, P, P, 1 << 20, None) == ESHAPE
    assert lib.moe4_grad_norm(None, None, None, 2, P, P, 1 << 20, None) == EINVAL
    assert clip([P], [4], [BF], [None]) == EINVAL and "outs[0] is NULL" in moe4.moe4_last_error()
    assert clip([P], [4], [BF], [MIS]) == EALIGN and "outs[0]" in moe4.moe4_last_error()
    assert clip([P], [4], [BF], mx=0.0) == EINVAL and "max_norm" in moe4.moe4_last_error()
    assert clip([P], [4], [BF], mx=float("nan")) == EINVAL
    assert clip([P], [4], [BF], ws=None) == EWS
    assert clip([P], [4], [BF], ni=P + 2) == EALIGN
    assert lib.moe4_grad_workspace_size(-1) == 0
    assert lib.moe4_grad_workspace_size(0) >= 256
    assert lib.moe4_grad_workspace_size(300) >= lib.moe4_grad_workspace_size(1)


def test_binding_refuses_what_the_kernels_cannot_read():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="GPU"):
        moe4.moe4_add_rmsnorm(x, x[0], 1e-6, out=x)
    with pytest.raises(TypeError, match="GPU"):
        moe4.moe4_quantize_mxfp8(x, x, x)
    with pytest.raises(TypeError, match="GPU"):
        moe4.GradList([x])
    with pytest.raises(ValueError, match="differ in length"):
        moe4.GradList([], [x])


def test_binding_refuses_sizes_past_int32():
    # cut off to 32 bits, 2^32 + 3 rows would be 3
    big = torch.empty(((1 << 32) + 3, 64), dtype=torch.bfloat16, device="meta")
    wide = torch.empty((1, (1 << 32) + 64), dtype=torch.bfloat16, device="meta")
    for x in (big, wide):
        with pytest.raises(ValueError, match="outside"):
            moe4.moe4_add_rmsnorm(x, x[0], 1e-6, out=x)
        with pytest.raises(ValueError, match="outside"):
            moe4.moe4_add_rmsnorm_backward(x, x, x[0], x[:, 0], x)
    with pytest.raises(ValueError, match="outside"):
        moe4.moe4_add_rmsnorm_workspace_size((1 << 32) + 3, 64)
    with pytest.raises(ValueError, match="I = 4294967360 outside"):
        moe4.Ffn(moe4.MOE4_FFN_BF16, wide, wide, gu_layout=1, act=1, H=64, I=(1 << 32) + 64)
    with pytest.raises(ValueError, match="T = 4294967299 outside"):
        moe4.moe4_ffn_workspace_size(None, (1 << 32) + 3)
