"""The sums of hc_build_block_tables (csrc/counts.h), compiled for the host
with g++: prefix sums in the kernel's grouping (4 requests to a thread, 32
lanes, 32 warps, chunk after chunk) against 64-bit sums cut off at 2^31 - 1
(CPU only)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <random>
#include <vector>
#include "counts.h"
using namespace hc;
static uint32_t cut(unsigned long long v) { return v < kMostCount ? (uint32_t)v : kMostCount; }
int main() {
  std::mt19937_64 rng(1);
  long bad = 0;
  for (int kind = 0; kind < 60; ++kind) {
    const int n = kind % 4 == 0 ? 1 + kind : kind % 4 == 1 ? 300 : kind % 4 == 2 ? 4096 : 9001;
    std::vector<uint32_t> tok(n), blk(n);
    for (int r = 0; r < n; ++r) {
      const unsigned odds = rng() % 100;
      tok[r] = odds < (unsigned)(kind % 7) * 5 ? kMostCount - rng() % 3 : rng() % 5000;
      blk[r] = odds >= 97 && kind % 3 == 0 ? kMostCount : rng() % 300;
    }
    unsigned long long st = 0, sb = 0;   // exact
    uint64_t carry = 0;
    for (int r0 = 0; r0 < n; r0 += 4096) {
      const int nr = n - r0 < 4096 ? n - r0 : 4096;
      std::vector<uint64_t> sum(1024), inc(1024), warp(32);
      auto value = [&](int r) { return r < nr ? counts(tok[r0 + r], blk[r0 + r]) : 0; };
      for (int t = 0; t < 1024; ++t)
        for (int i = 0; i < 4; ++i) sum[t] = add_counts(sum[t], value(4 * t + i));
      auto scan = [](std::vector<uint64_t> v, int at) {   // the doubling scan of 32 lanes from `at`
        for (int o = 1; o < 32; o <<= 1) {
          std::vector<uint64_t> w = v;
          for (int l = o; l < 32; ++l) w[at + l] = add_counts(v[at + l], v[at + l - o]);
          v = w;
        }
        return v;
      };
      inc = sum;
      for (int w = 0; w < 32; ++w) inc = scan(inc, 32 * w), warp[w] = inc[32 * w + 31];
      warp = scan(warp, 0);
      for (int t = 0; t < 1024; ++t) {
        const uint64_t before = t % 32 ? inc[t - 1] : 0, warps = t / 32 ? warp[t / 32 - 1] : 0;
        uint64_t at = add_counts(carry, add_counts(warps, before));
        for (int i = 0; i < 4; ++i) {
          const int r = 4 * t + i;
          if (r >= nr) break;
          bad += tokens_of(at) != cut(st) || blocks_of(at) != cut(sb);
          st += tok[r0 + r], sb += blk[r0 + r];
          at = add_counts(at, value(r));
        }
      }
      carry = add_counts(carry, warp[31]);
      bad += tokens_of(carry) != cut(st) || blocks_of(carry) != cut(sb);
    }
  }
  std::printf("%ld\n", bad);
  return bad != 0;
}
"""


def test_prefix_sums_stop_at_the_largest_count(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    src, exe = tmp_path / "t.cc", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-O2", "-std=c++17", "-I", os.path.join(ROOT, "kv_cache_quantization_hc_gb300", "csrc"), str(src),
                    "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "0", r.stdout + r.stderr


def test_counts_that_leave_no_room_are_refused():
    """Arrays of 2^31 - 1 entries: a sum that stopped there would not be seen to be too large."""
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from kv_cache_quantization_hc_gb300 import build, hc
    build.build()
    from tests.test_serve_refusals import _tables
    most = 2 ** 31 - 1
    assert _tables(hc, n_tokens=most) == hc.HC_ERR_INVALID_ARG
    assert _tables(hc, n_free=most) == hc.HC_ERR_INVALID_ARG
