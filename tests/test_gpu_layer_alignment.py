"""The layer for few tokens on tensors that begin where moe4.h allows it and an allocator rarely puts
them: scales in bytes at any address, fp32 arrays at 4 bytes, biases at 2."""
import numpy as np
import pytest
import torch

from gpu_helpers import to_dev
from test_gpu_dense import BF, draw, rng
from test_gpu_layer_decode import ALPHA, FMT, LIMIT, Stacks, moe4

pytestmark = pytest.mark.gpu


def moved(t, by):
    """A copy of t that begins `by` bytes past 256-byte aligned memory, between bytes of ones"""
    if t is None:
        return None
    n = t.numel() * t.element_size()
    raw = torch.full((n + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    at = 256 - raw.data_ptr() % 256 + by
    raw[at:at + n].copy_(t.contiguous().view(-1).view(torch.uint8))
    return raw[at:at + n].view(t.dtype).view(t.shape)


@pytest.mark.parametrize("T,E,k,H,I", [(1, 5, 3, 96, 160), (9, 5, 3, 96, 160), (32, 18, 16, 416, 480)])
@pytest.mark.parametrize("fmt", ["mx4", "nf4", "dq"])
def test_least_aligned_tensors(fmt, T, E, k, H, I):
    if fmt != "mx4":
        H, I = H // 64 * 64 + 64, I // 64 * 64
    st = Stacks("align", fmt, E, H, I, "interleaved", "clamped", True)
    x, _ = draw(rng("align x", T), (T, H))
    lg = to_dev(rng("align lg", T).standard_normal((T, E)).astype(np.float32))
    want = torch.empty((T, H), dtype=BF, device="cuda")
    moe4.moe4_layer_decode(st.ex, x, lg, k, want, ws=st.ws(T, k))
    gu_q, gu_s, dn_q, dn_s, gu_b, dn_b = st.ex.tensors[:6]
    desc, book = st.ex.desc, dict(zip(("gu_s2", "dn_s2", "gu_soff", "dn_soff", "dq_book"), st.ex.tensors[8:]))
    for by in (4, 8, 12) if fmt == "nf4" else (1, 2, 3):
        ex = moe4.Experts(FMT[fmt], gu_q, moved(gu_s, by), dn_q, moved(dn_s, by), E=E, H=H, I=I, gu_layout=desc.gu_layout,
                          act=desc.act, act_alpha=ALPHA, act_limit=LIMIT, gu_bias=moved(gu_b, 2), dn_bias=moved(dn_b, 6),
                          **{n: moved(t, 4) for n, t in book.items()})
        out = torch.empty_like(want)
        idx, w = moved(torch.zeros((T, k), dtype=torch.int32, device="cuda"), 4), moved(torch.zeros((T, k), device="cuda"), 12)
        moe4.moe4_layer_decode(ex, x, moved(lg, 4), k, out, topk_idx=idx, topk_w=w, ws=st.ws(T, k))
        assert torch.equal(out, want), by
