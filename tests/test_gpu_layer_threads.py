"""moe4_layer_decode from two host threads at once, with sizes that take different amounts of LDS."""
import threading

import pytest
import torch

from gpu_helpers import to_dev
from test_gpu_dense import BF, draw, rng
from test_gpu_layer_decode import Stacks, moe4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["nf4", "mx4", "dq"])
def test_two_threads_with_different_sizes(fmt):
    # T, E, k: from a few KB of LDS beside the table, and of activations, to the most slots
    jobs = []
    for T, E, k in ((1, 4, 1), (32, 64, 16)):
        st = Stacks("threads", fmt, E, 1024, 64)
        x, _ = draw(rng("thread x", T), (T, 1024))
        lg = to_dev(rng("thread lg", T).standard_normal((T, E)).astype("float32"))
        want, out = (torch.empty((T, 1024), dtype=BF, device="cuda") for _ in range(2))
        ws = st.ws(T, k)
        moe4.moe4_layer_decode(st.ex, x, lg, k, want, ws=ws)
        jobs.append((st, x, lg, k, want, out, ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    start, errors = threading.Barrier(2), []

    def work(st, x, lg, k, want, out, ws, stream):
        try:
            start.wait()
            for i in range(200):
                if i % 50 == 0:
                    with torch.cuda.stream(stream):
                        out.fill_(float("nan"))
                moe4.moe4_layer_decode(st.ex, x, lg, k, out, ws=ws, stream=stream)
                if i % 50 == 49:
                    stream.synchronize()
                    assert torch.equal(out.cpu(), want.cpu()), i
        except BaseException as e:   # noqa: BLE001 (handed to the test's thread)
            errors.append(e)
    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
