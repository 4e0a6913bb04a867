"""Waits on barriers that nobody arrives at end with a status, and the context stays usable
(csrc/mbarrier.cuh, in a kernel of its own: two warps wait for nothing, a third for an arrival)."""
import ctypes
import os
import subprocess
import time

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include "mbarrier.cuh"
using namespace hc;
__global__ void k_wait(int32_t* out) {
  __shared__ uint64_t bars[3];
  __shared__ int32_t dead;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 3; ++i) mbar_init(&bars[i], 1);
    dead = 0;
  }
  __syncthreads();
  if (threadIdx.x == 64) mbar_arrive(&bars[2]);
  const bool there = mbar_wait(&bars[warp], 0, &dead);
  if ((threadIdx.x & 31) == 0) out[warp] = there;
  __syncthreads();
  if (threadIdx.x == 0) out[3] = dead;
}
extern "C" int run_wait(int32_t* out, void* stream) {
  k_wait<<<1, 96, 0, static_cast<cudaStream_t>(stream)>>>(out);
  return cudaGetLastError();
}
"""


def test_waits_end(tmp_path):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from kv_cache_quantization_hc_gb300 import build
    src, lib = tmp_path / "wait.cu", tmp_path / "wait.so"
    src.write_text(PROGRAM)
    subprocess.run([build._nvcc(), *build.FLAGS, "-I", build.CSRC, "-shared", str(src), "-o", str(lib)], check=True)
    run = ctypes.CDLL(str(lib)).run_wait
    run.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    out = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    start = time.monotonic()
    assert run(out.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    took = time.monotonic() - start
    assert out.tolist() == [0, 0, 1, 1]
    assert 1.9 < took < 4, took                  # the second of the two did not start its own two seconds after the first's
    assert float(torch.ones(5, device="cuda").sum()) == 5
