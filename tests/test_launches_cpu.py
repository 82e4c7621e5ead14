"""Grids, LDS and workspaces of the launches, without a GPU."""
import math
import random

import pytest

from tests.launches import LDS, first_lds, record, second_cut, table_lds

moe4 = pytest.importorskip("bit_mixture_experts_amd.moe4")

P = 0x10000000   # 256-byte aligned, never dereferenced
FMT = {"nf4": moe4.MOE4_FMT_NF4, "mx4": moe4.MOE4_FMT_MXFP4, "dq": moe4.MOE4_FMT_NF4_DQ}
BF = moe4.MOE4_DTYPE_BF16

# fmt, T, E, k, H, I: few and many tokens, experts, units; activations that fit LDS and that do not
LAYERS = [("nf4", 1, 128, 8, 2048, 768), ("nf4", 16, 128, 8, 2048, 768), ("nf4", 32, 1024, 16, 64, 64),
          ("nf4", 4, 4, 2, 64, 64), ("dq", 1, 16, 2, 2048, 768), ("dq", 32, 512, 16, 4096, 1024),
          ("mx4", 1, 32, 4, 2880, 2880), ("mx4", 8, 32, 4, 2880, 2880), ("mx4", 27, 32, 4, 2880, 32),
          ("mx4", 28, 32, 4, 2880, 32), ("mx4", 32, 32, 4, 2880, 288), ("mx4", 32, 300, 4, 2880, 96),
          ("mx4", 2, 300, 8, 64, 32), ("mx4", 32, 1024, 16, 8192, 32), ("mx4", 32, 8, 2, 1 << 20, 32)]


def layer_call(fmt, T, E, k, H, I):
    d = dict(struct="Moe4Experts", format=FMT[fmt], E=E, H=H, I=I, gu_layout=1, act=1, act_alpha=1.702, act_limit=7.0,
             gu_q=P, gu_s=P, dn_q=P, dn_s=P)
    if fmt == "dq":
        d.update(gu_s2=P, dn_s2=P, gu_soff=P, dn_soff=P, dq_book=P)
    return ["moe4_layer_decode", [d, P, P, T, k, 1, None, 0, P, BF, None, None, P, 1 << 30, None]]


def linear_calls():
    for T in (1, 9, 16, 17, 32, 33, 64, 500, 3000):
        for N, K in ((64, 64), (4096, 4096), (16384, 2048)):
            lin = dict(struct="Moe4Linear", N=N, K=K, variant=0, w_q=P, w_s=P)
            for f in (moe4.MOE4_X_BF16, moe4.MOE4_X_MXFP8, moe4.MOE4_X_MXFP4):
                yield ["moe4_linear_forward", [dict(lin), P, f, None if f == moe4.MOE4_X_BF16 else P, T, None, 0, P, BF, P,
                                               1 << 40, None]]
            yield ["moe4_linear_backward", [dict(lin), P, T, None, 0, P, BF, P, BF, P, 1 << 40, None]]


@pytest.fixture(scope="module")
def recorded(tmp_path_factory):
    calls = [layer_call(*c) for c in LAYERS] + list(linear_calls())
    got = record(calls, tmp_path_factory.mktemp("rec"))
    assert all(r["rc"] == 0 for r in got), [r["error"] for r in got if r["rc"]]
    return got


def test_the_most_lds_of_a_kernel_is_one_number(recorded):
    # It is the process's setting: a call that lowered it to its own need would have another thread's
    # launch, between setting and launching, refused.
    most, launches = {}, 0
    for r in recorded:
        for e in r["events"]:
            if e["allowed"] >= 0:
                most.setdefault(e["kernel"], set()).add(e["allowed"])
            else:
                launches += 1
                allowed = max(most.get(e["kernel"], {65536}))
                assert e["lds"] <= allowed <= LDS, (e, allowed)
    assert launches >= 2 * len(LAYERS)
    assert all(len(v) == 1 for v in most.values()), most


def test_the_layer_launches_what_its_rules_say(recorded):
    inside, cuts = set(), set()
    for (fmt, T, E, k, H, I), r in zip(LAYERS, recorded):
        up, down = [e for e in r["events"] if e["allowed"] < 0]
        lds, x = first_lds(fmt, T, E, k, H)
        assert up["lds"] == lds and up["grid"] == [min(T * k * (I // 4), 256), 1, 1] and up["block"][0] == 512
        cut, each = second_cut(fmt, T, k, H, I)
        assert down["lds"] == table_lds(fmt) + 2048 * (2 if cut else 1) + 16 * T * k + 4
        assert down["grid"] == [256 if cut else H // 8 * -(-T // 8), 1, 1] and down["block"][0] == 512
        inside.add((fmt, x))
        cuts.add((fmt, cut))
    assert inside == {("nf4", False), ("dq", False), ("mx4", False), ("mx4", True)}
    assert cuts == {(f, c) for f in FMT for c in (False, True)}


def test_parts_of_linear_products_fit_the_workspace(tmp_path):
    # a product cut along k leaves `splits` sums of all its outputs: read off the grid, for drawn sizes
    r = random.Random(7)
    size = lambda lo, hi, m: max(m, round(math.exp(r.uniform(math.log(lo), math.log(hi)))) // m * m)   # noqa: E731
    calls, what = [], []
    while len(what) < 400:
        N, K, T = size(8, 30000, 8), size(32, 30000, 32), size(1, 20000, 1)
        lin = dict(struct="Moe4Linear", N=N, K=K, variant=r.choice([0, moe4.MOE4_VARIANT_TILED]), w_q=P, w_s=P)
        f = r.choice([moe4.MOE4_X_BF16, moe4.MOE4_X_MXFP8, moe4.MOE4_X_MXFP4])
        calls += [["moe4_linear_workspace_size", [dict(lin), T, 0]],
                  ["moe4_linear_forward", [dict(lin), P, f, None if f == moe4.MOE4_X_BF16 else P, T, None, 0, P, BF, P, 1 << 40, None]],
                  ["moe4_linear_workspace_size", [dict(lin), T, 1]],
                  ["moe4_linear_backward", [dict(lin), P, T, None, 0, P, BF, P, BF, P, 1 << 40, None]]]
        what += [(N, T, 64, 0), (K, T, 128, 128 * N * 4 if T > 512 else 0)]   # outputs, rows, rows of a tile, more
    got, cut = record(calls, tmp_path), 0
    for (cols, rows, tile, more), bytes_, call in zip(what, got[0::2], got[1::2]):
        assert call["rc"] == 0
        first = [e for e in call["events"] if e["allowed"] < 0][0]
        tiles = -(-cols // 128) * -(-rows // tile)
        if first["block"][0] != 256 or first["grid"][1] != 1:
            continue   # few tokens, or the larger tiles, which are not cut
        splits, rest = divmod(first["grid"][0], tiles)
        assert rest == 0 and splits >= 1
        part = splits * rows * cols * 4 if splits > 1 else 0
        assert (-(-part // 256) * 256 + more if more else part) <= bytes_["rc"], (cols, rows, splits)
        cut += splits > 1
    assert cut > 50
