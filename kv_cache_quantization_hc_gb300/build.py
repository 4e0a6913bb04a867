"""Build libhc.so (the C-ABI library) in-tree with nvcc for sm_103a, and,
where torch is installed, _serve (the Python binding of the serving calls,
over torch's C++ headers) with the host compiler.

The translation units compile in parallel; the link uses nvcc's default
static CUDA runtime, so the library depends on no libcudart at load time.
A stamp of the sources' hash and the flags skips rebuilding an up-to-date
library built for this machine's architecture.
"""
import fcntl
import hashlib
import importlib.util
import os
import platform
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libhc.so")
BINDING = os.path.join(PKG, "_serve" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))

SOURCES = ["api.cu", "encode.cu", "encode_rows.cu", "fetch_fp8.cu", "fetch_fp8_rows.cu",
           "fetch_int4.cu", "fetch_raw.cu", "table.cu", "crc32.cu", "select.cu",
           "api_serve.cu", "block_tables.cu", "rope_axes.cu", "append.cu", "attend.cu",
           "attend_tiles.cu", "api_paged.cu", "append_paged.cu", "attend_paged.cu",
           "attend_paged_tiles_64.cu", "attend_paged_tiles_128.cu", "merge.cu",
           "hash.cpp"]


def _headers():
    """Every header the translation units may include: all of csrc/'s, and hc.h."""
    hs = sorted(f for f in os.listdir(CSRC) if f.endswith((".h", ".cuh")))
    return [os.path.join(CSRC, h) for h in hs] + [os.path.join(INCLUDE, "hc.h")]


ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE]

_ELF_MACHINE = {"x86_64": 62, "aarch64": 183, "arm64": 183}


def _nvcc():
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libhc.so")


def _binding_flags():
    """(compile, link) flags of the binding: torch's headers and libraries,
    Python's and the toolkit's headers, and libhc.so beside it."""
    import torch
    home = os.path.dirname(torch.__file__)
    inc = [INCLUDE, os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")]
    lib = os.path.join(home, "lib")
    flags = ["-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for d in inc:
        flags += ["-isystem", d]
    return flags, ["-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-ltorch",
                   "-L", PKG, "-l:libhc.so", f"-Wl,-rpath,{lib}", "-Wl,-rpath,$ORIGIN"]


def _digest(paths, *words):
    h = hashlib.sha256()
    for p in paths:
        with open(p, "rb") as f:
            h.update(p.encode() + b"\0" + f.read())
    for w in words + (platform.machine(),):
        h.update(w.encode() + b"\0")
    return h.hexdigest()


def _stamp(extra_flags):
    return _digest([os.path.join(CSRC, s) for s in SOURCES] + _headers(), " ".join(FLAGS + list(extra_flags)))


def _torch_home():
    """Where torch is installed, found without importing it; None where it is not."""
    spec = importlib.util.find_spec("torch")
    return None if spec is None or spec.origin is None else os.path.dirname(spec.origin)


def _binding_stamp(torch_home):
    return _digest([os.path.join(CSRC, "binding.cpp"), os.path.join(INCLUDE, "hc.h"),
                    os.path.join(torch_home, "version.py")], sys.version)


def _current(path, stamp_path, stamp):
    """True if the file at path was built here for this stamp."""
    if not _lib_matches_host(path) or not os.path.exists(stamp_path):
        return False
    with open(stamp_path) as f:
        return f.read().strip() == stamp


def _lib_matches_host(path):
    """True if the ELF at path was built for this machine's architecture."""
    try:
        with open(path, "rb") as f:
            hdr = f.read(20)
    except OSError:
        return False
    if len(hdr) < 20 or hdr[:4] != b"\x7fELF":
        return False
    machine = int.from_bytes(hdr[18:20], "little")
    return machine == _ELF_MACHINE.get(platform.machine(), -1)


def build(force=False, verbose=False, extra_flags=(), out_dir=None):
    """Compile and link libhc.so, and where torch is installed the binding;
    returns the library's path.  ``out_dir`` places the objects and the
    library elsewhere (a variant built with extra flags, without a binding).
    Concurrent callers (the ranks of a torchrun job) take turns on a lock
    file in the build directory: the first builds, the others then find the
    stamp up to date."""
    build_dir = BUILD if out_dir is None else out_dir
    os.makedirs(build_dir, exist_ok=True)
    with open(os.path.join(build_dir, "lock"), "w") as lock:
        fcntl.flock(lock, fcntl.LOCK_EX)
        try:
            return _build_locked(build_dir, force, verbose, extra_flags, out_dir)
        finally:
            fcntl.flock(lock, fcntl.LOCK_UN)


def _run(what, cmd, verbose=False):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr)


def _build_library(lib, build_dir, verbose, extra_flags, ex):
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(build_dir, os.path.splitext(src)[0] + ".o")
        _run(f"nvcc on {src}", [nvcc, *FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj], verbose)
        return obj

    objs = list(ex.map(compile_one, SOURCES))
    _run("link", [nvcc, *ARCH, "-shared", "-o", lib + ".tmp", *objs])
    os.replace(lib + ".tmp", lib)


def _compile_binding(build_dir):
    """Compiles it; the command that links it, once libhc.so is there, without its output."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        raise RuntimeError("a C++ compiler is required to build the Python binding")
    flags, libs = _binding_flags()
    obj = os.path.join(build_dir, "binding.o")
    _run("binding", [cxx, *flags, "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj])
    return [cxx, "-shared", obj, *libs]


def _build_locked(build_dir, force, verbose, extra_flags, out_dir):
    lib = LIB if out_dir is None else os.path.join(out_dir, "libhc.so")
    stamp, stamp_path = _stamp(extra_flags), os.path.join(build_dir, "stamp")
    binding_stamp_path = os.path.join(build_dir, "binding_stamp")
    # the library needs nvcc alone; the binding is for torch's tensors
    torch_home = _torch_home() if out_dir is None else None
    with_binding = torch_home is not None
    binding_stamp = _binding_stamp(torch_home) if with_binding else None
    library_due = force or not _current(lib, stamp_path, stamp)
    binding_due = with_binding and (force or not _current(BINDING, binding_stamp_path, binding_stamp))
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding, build_dir) if binding_due else None
        if library_due:
            _build_library(lib, build_dir, verbose, extra_flags, ex)
            with open(stamp_path, "w") as f:
                f.write(stamp)
        if binding_due:
            _run("binding's link", binding.result() + ["-o", BINDING + ".tmp"])
            os.replace(BINDING + ".tmp", BINDING)
            with open(binding_stamp_path, "w") as f:
                f.write(binding_stamp)
    return lib


if __name__ == "__main__":
    print(build(force=True, verbose=True))
