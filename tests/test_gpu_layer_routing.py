"""The routing inside the layer for few tokens against moe4_route: one order of experts, NaNs among them."""
import numpy as np
import pytest
import torch

from gpu_helpers import to_dev
from test_gpu_dense import BF, U32, rng
from test_gpu_layer_decode import Stacks, moe4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 64, 8), (1, 1024, 70), (32, 70, 16), (32, 300, 16), (7, 1024, 73), (5, 3, 3)])
def test_the_layer_routes_as_moe4_route(T, E, k, renorm):
    st = Stacks("routing", "nf4", E, 64, 64)
    r = rng("routing", T, E)
    lg = r.choice(np.array([0.0, -0.0, 1e-45, -1e-45, 0.5, -0.5, 2.0, 3e38, -3e38, -np.inf], np.float32), (T, E))
    if T > 1:
        lg[T // 2:] = r.standard_normal((T - T // 2, E))
        lg[T // 2, ::2] = np.nan     # half of the experts, which come last, the lower first
        lg[T - 1, 1:] = -np.inf
    x, logits = torch.zeros((T, 64), dtype=BF, device="cuda"), to_dev(lg)
    out = torch.empty((T, 64), dtype=BF, device="cuda")
    idx = [torch.full((T, k), -1, dtype=torch.int32, device="cuda") for _ in range(2)]
    w = [torch.full((T, k), -1.0, device="cuda") for _ in range(2)]
    moe4.moe4_route(logits, k, idx[0], w[0], renormalize=renorm)
    moe4.moe4_layer_decode(st.ex, x, logits, k, out, topk_idx=idx[1], topk_w=w[1], renormalize=renorm, ws=st.ws(T, k))
    assert torch.equal(idx[0], idx[1])
    a, b = (v.double().cpu().numpy() for v in w)
    assert np.array_equal(np.isnan(a), np.isnan(b))
    # the same quotients, with sums of k or E terms in another order
    ok = ~np.isnan(a)
    assert np.all(np.abs(a[ok] - b[ok]) <= 2 * (E + 4) * U32 * np.abs(a[ok]))
