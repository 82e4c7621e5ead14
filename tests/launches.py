"""What a call of the library would launch, seen without a GPU: launch_recorder.cpp stands in for HIP's
launch functions in a child interpreter. And the rules by which moe4_layer_decode picks its kernels, as
tests state them (tests/test_launches_cpu.py holds them against what is launched)."""
import json
import os
import subprocess
import sys

from tests.conftest import ROOT

# the child: calls = [[function, arguments]]; a dict among the arguments is a descriptor
CHILD = """
import ctypes, json, sys
rec = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
from bit_mixture_experts_amd import moe4
class Event(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_void_p), ("grid", ctypes.c_uint32 * 3), ("block", ctypes.c_uint32 * 3),
                ("lds", ctypes.c_int64), ("allowed", ctypes.c_int64)]
ev = (Event * 4096)()
out = []
for fn, args in json.load(sys.stdin):
    args = [ctypes.byref(getattr(moe4, a.pop("struct"))(**a)) if isinstance(a, dict) else a for a in args]
    rec.recorder_take(ev)
    rc = getattr(moe4._lib, fn)(*args)
    n = rec.recorder_take(ev)
    out.append(dict(rc=rc, error=moe4.moe4_last_error() if rc else "", events=[
        dict(kernel=e.kernel, grid=list(e.grid), block=list(e.block), lds=e.lds, allowed=e.allowed) for e in ev[:n]]))
print("EVENTS" + json.dumps(out))
"""


def record(calls, tmp_path):
    """[dict(rc, error, events)] of the calls, in their order"""
    lib = str(tmp_path / "librecorder.so")
    subprocess.run(["g++", "-O1", "-shared", "-fPIC", os.path.join(ROOT, "tests", "launch_recorder.cpp"), "-o", lib],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([sys.executable, "-c", CHILD, lib], input=json.dumps(calls), cwd=ROOT, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    return json.loads(r.stdout.split("EVENTS")[1])


# ---- the rules of moe4_layer_decode

LDS = 160 * 1024


def table_lds(fmt):
    return {"mx4": 0, "nf4": 65536, "dq": 65536 + 1024}[fmt]


def first_lds(fmt, T, E, k, H):
    """(dynamic LDS of the first launch, whether the activations are in it)"""
    n = -(-(table_lds(fmt) + 8 * E + 20 * T * k + 4) // 16) * 16
    x = T * (2 * H + 32)
    inside = fmt == "mx4" and n + x <= LDS
    return n + (x if inside else 0), inside


def second_cut(fmt, T, k, H, I):
    """whether the second launch cuts its panels, and how many steps of 256 a unit has"""
    most, steps = 4 if fmt == "mx4" else 3, -(-I // 256)
    runs = -(-steps // most)
    each = -(-steps // runs)
    return H // 16 * T * k * -(-steps // each) >= 12288, each
