"""libhc.so is built where torch is not installed, as for a C client, and the
binding where it is (CPU only; one small source stands for all of them)."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
import ctypes, os, sys
sys.path.insert(0, {root!r})
if {hide}:
    sys.modules["torch"] = None
from kv_cache_quantization_hc_gb300 import build
build.SOURCES = ["hash.cpp"]
build.BUILD, build.PKG = {out!r}, {out!r}
build.LIB = os.path.join({out!r}, "libhc.so")
build.BINDING = os.path.join({out!r}, os.path.basename(build.BINDING))
built = []
compile_binding = build._compile_binding
build._compile_binding = lambda d: built.append(d) or ["true"]
try:
    lib = build.build()
except FileNotFoundError:      # no binding came of the stand-in
    lib = build.LIB
ctypes.CDLL(lib).hc_block_digests
when = os.path.getmtime(lib)
if {hide}:
    assert build.build() == lib and os.path.getmtime(lib) == when    # up to date
print(len(built))
"""


@pytest.mark.parametrize("hide", [True, False])
def test_build(tmp_path, hide):
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    r = subprocess.run([sys.executable, "-c", PROGRAM.format(root=ROOT, hide=hide, out=str(tmp_path))], capture_output=True,
                       text=True, timeout=300, cwd=str(tmp_path))
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.split()[-1] == ("0" if hide else "1")
