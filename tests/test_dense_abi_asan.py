"""The dense operators' argument validation under AddressSanitizer, without a GPU: a child
interpreter loads libmoe4_asan.so (the C entry points with ASan on their host code) and runs
test_dense_abi_cpu.py, whose calls read descriptors and host arrays of every size."""
import os
import subprocess
import sys

from tests.conftest import ROOT
from tests.test_abi_asan import LIB, _asan_runtime


def test_dense_validation_runs_clean_under_asan():
    assert os.path.exists(LIB), "libmoe4_asan.so is not built"
    runtime = _asan_runtime()
    assert runtime, "the ROCm clang ASan runtime is missing"
    env = dict(os.environ, MOE4_LIB_PATH=LIB,
               ASAN_OPTIONS="detect_leaks=0:exitcode=86:halt_on_error=1",
               LD_PRELOAD=":".join(p for p in (runtime, os.environ.get("LD_PRELOAD", "")) if p))
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                        "-m", "not gpu", os.path.join(ROOT, "tests", "test_dense_abi_cpu.py")],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out, out[-4000:]
    assert r.returncode == 0, out[-4000:]
    assert " passed" in r.stdout
