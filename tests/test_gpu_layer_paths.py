"""Parity of the routed layer for few tokens on each kernel that it picks, by the rules of
tests/launches.py (held against the launches themselves in tests/test_launches_cpu.py)."""
import pytest

from launches import first_lds, second_cut
from test_gpu_dense import BF, F32
from test_gpu_layer_decode import Stacks, check

pytestmark = pytest.mark.gpu


# MXFP4 with the tokens' activations in LDS, and not, where they do not fit: up to and beyond 128 experts,
# one, two and more tiles to a wave, rows of an expert in several passes of 8, one token
@pytest.mark.parametrize("inside,T,E,k,H,I,layout,bias", [
    (True, 27, 32, 4, 2880, 32, "halves", True), (False, 28, 32, 4, 2880, 32, "halves", True),
    (True, 19, 40, 6, 4096, 64, "interleaved", False), (False, 20, 40, 6, 4096, 64, "interleaved", False),
    (False, 32, 32, 4, 2880, 288, "interleaved", True), (False, 32, 300, 4, 2880, 96, "halves", True),
    (False, 32, 300, 16, 2880, 32, "interleaved", True), (False, 32, 16, 16, 2880, 416, "halves", True),
    (False, 32, 16, 16, 2912, 416, "interleaved", False), (False, 32, 2, 2, 3104, 672, "halves", False),
    (False, 1, 3, 2, 90112, 32, "halves", True), (False, 2, 140, 3, 49152, 32, "interleaved", False)])
def test_activations_in_lds_and_not(inside, T, E, k, H, I, layout, bias):
    assert first_lds("mx4", T, E, k, H)[1] == inside
    check(Stacks("lds", "mx4", E, H, I, layout, "clamped" if bias else "swiglu", bias), T, k, renorm=T != 20,
          res=(None, BF, F32)[T % 3])


# the second launch with its panels cut from 12288 units on, and whole: units of up to two, three and four steps
@pytest.mark.parametrize("fmt,T,E,k,H,I,cut,steps", [
    ("nf4", 32, 24, 16, 384, 64, True, 1), ("nf4", 32, 24, 16, 320, 64, False, 1),
    ("nf4", 9, 64, 8, 2112, 832, True, 2), ("nf4", 8, 32, 8, 4096, 768, True, 3), ("nf4", 7, 32, 8, 2048, 768, False, 3),
    ("nf4", 31, 12, 8, 448, 960, True, 2), ("nf4", 12, 20, 8, 1024, 576, False, 3),
    ("mx4", 17, 300, 30, 416, 32, True, 1), ("mx4", 32, 24, 16, 352, 480, False, 2), ("mx4", 32, 24, 16, 384, 480, True, 2),
    ("mx4", 32, 16, 16, 416, 704, True, 3), ("mx4", 32, 16, 16, 352, 704, False, 3), ("mx4", 32, 16, 16, 416, 1024, True, 4),
    ("mx4", 9, 16, 16, 416, 1024, False, 4), ("dq", 32, 16, 16, 384, 448, True, 2), ("dq", 32, 16, 16, 320, 448, False, 2),
    ("dq", 30, 16, 16, 448, 640, True, 3), ("dq", 5, 16, 16, 448, 640, False, 3)])
def test_panels_cut_and_whole(fmt, T, E, k, H, I, cut, steps):
    assert second_cut(fmt, T, k, H, I) == (cut, steps)
    bias = T % 2 == 1
    check(Stacks("cut", fmt, E, H, I, "interleaved" if bias else "halves", "clamped" if bias else "swiglu", bias), T, k,
          res=(BF, F32, None)[T % 3])
