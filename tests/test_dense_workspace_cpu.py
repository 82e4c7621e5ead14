"""Workspace sizes of the dense operators: one buffer made for the largest batch serves every
smaller one, so no size falls as the number of tokens grows. Nothing here reaches a device."""
import ctypes

import pytest

moe4 = pytest.importorskip("bit_mixture_experts_amd.moe4")
lib = moe4._lib
P = 0x10000   # 256-byte aligned, never dereferenced

# the smallest blocks, ordinary ones, a long reduction, a wide stream
SIZES = [(8, 8), (64, 96), (1024, 128), (2048, 768), (2880, 2880), (4096, 8192), (4104, 136), (8192, 32), (32, 8192)]


def _sizes_of_t():
    t = set(range(0, 2100)) | set(range(2100, 9000, 37))
    for k in range(1, 520):   # both sides of every row tile
        t |= {128 * k - 1, 128 * k, 128 * k + 1}
    return sorted(t)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("H,I", SIZES)
def test_block_sizes_never_fall(H, I, mx):
    if mx and (H % 32 or I % 32):
        H, I = -(-H // 32) * 32, -(-I // 32) * 32
    d = moe4.Moe4Ffn(format=moe4.MOE4_FFN_MXFP8 if mx else moe4.MOE4_FFN_BF16, H=H, I=I, gu_layout=moe4.MOE4_GU_HALVES,
                     act=moe4.MOE4_ACT_SWIGLU, act_alpha=1.702, act_limit=7.0, variant=0, w_gu=P, w_dn=P,
                     gu_s=P if mx else None, dn_s=P if mx else None)
    for backward in (0, 1):
        last = 0
        for T in _sizes_of_t():
            n = lib.moe4_ffn_workspace_size(ctypes.byref(d), T, backward)
            assert n >= last > 0 or (last == 0 and n > 0), (T, backward, n, last)
            last = n


@pytest.mark.parametrize("H,I", [(64, 96), (2048, 768), (2880, 2880), (4096, 8192)])
def test_block_sizes_are_not_extravagant(H, I):
    # what a call holds (h; dGU and h), its partial sums (at most 512 tiles of 64 KiB along k, and
    # in the backward pass twice, with the biases' sums beside them), and alignment
    d = moe4.Moe4Ffn(format=moe4.MOE4_FFN_BF16, H=H, I=I, gu_layout=moe4.MOE4_GU_HALVES, act=moe4.MOE4_ACT_SWIGLU,
                     act_alpha=1.702, act_limit=7.0, variant=0, w_gu=P, w_dn=P)
    for T in (1, 100, 1024, 8192, 100000):
        fwd, bwd = (lib.moe4_ffn_workspace_size(ctypes.byref(d), T, b) for b in (0, 1))
        assert fwd <= T * I * 2 + (32 << 20) + 4096
        sums = 2 * I * 4 * max(-(-T // 128), min(-(-T // 16), 2048)) + 128 * max(H, 2 * I) * 4
        assert bwd <= T * I * 6 + sums + (64 << 20) + 8192


@pytest.mark.parametrize("H", [8, 512, 520, 1024, 2048, 2056, 2880, 4096, 4104, 8192, 16384])
def test_norm_sizes_never_fall(H):
    last = 0
    for T in _sizes_of_t() + [1 << 17, 1 << 20, 1 << 30]:
        n = lib.moe4_add_rmsnorm_workspace_size(T, H)
        assert n >= last and n > 0, (T, n, last)
        last = n


def test_grad_sizes_never_fall():
    last = 0
    for n in list(range(0, 1000)) + [1 << k for k in range(10, 21)]:
        size = lib.moe4_grad_workspace_size(n)
        assert size >= last and size > 0
        last = size
