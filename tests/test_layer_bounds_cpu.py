"""Bounds of moe4_layer_decode that moe4.h states: the widest rows of each format."""
import ctypes

import pytest

moe4 = pytest.importorskip("bit_mixture_experts_amd.moe4")
P = 0x10000
DQ = dict(gu_s2=P, dn_s2=P, gu_soff=P, dn_soff=P, dq_book=P)


@pytest.mark.parametrize("fmt,H,I,code,msg", [
    (moe4.MOE4_FMT_NF4, 1 << 20, 64, 0, ""), (moe4.MOE4_FMT_MXFP4, 1 << 20, 32, 0, ""),
    (moe4.MOE4_FMT_NF4, 64, 1 << 19, 0, ""), (moe4.MOE4_FMT_NF4_DQ, 16384, 16384, 0, ""),
    (moe4.MOE4_FMT_NF4, (1 << 20) + 64, 64, moe4.MOE4_ESHAPE, "beyond 2^20"),
    (moe4.MOE4_FMT_MXFP4, (1 << 20) + 32, 32, moe4.MOE4_ESHAPE, "beyond 2^20"),
    (moe4.MOE4_FMT_NF4_DQ, 16448, 64, moe4.MOE4_EUNSUPPORTED, "16384"),
    (moe4.MOE4_FMT_NF4_DQ, 64, 16448, moe4.MOE4_EUNSUPPORTED, "16384")])
def test_widest_rows(fmt, H, I, code, msg):
    ex = moe4.Moe4Experts(format=fmt, E=4, H=H, I=I, gu_layout=1, act=1, gu_q=P, gu_s=P, dn_q=P, dn_s=P,
                          **(DQ if fmt == moe4.MOE4_FMT_NF4_DQ else {}))
    size = moe4._lib.moe4_layer_decode_workspace_size(ctypes.byref(ex), 32, 4)
    assert (size > 0) == (code == 0)
    if code:
        assert msg in moe4.moe4_last_error()
