"""The rule between the two attention kernels, asked on the host (CPU only)."""
import os
import shutil

import pytest


@pytest.fixture(scope="module")
def few():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from kv_cache_quantization_hc_gb300 import build, hc
    build.build()
    return hc.lib().hc_attend_int4_few_rows


def test_limits(few):
    """Whole pieces of 16 rows, 384 at most, 16 at least, and no more with more requests to share the GPU."""
    for d in (64, 128):
        for heads in (1, 2, 8, 40):
            rows = [few(n, heads, d) for n in (1, 2, 4, 16, 64, 256, 4096, 1 << 20)]
            assert all(r % 16 == 0 and 16 <= r <= 384 for r in rows) and rows == sorted(rows, reverse=True)
    assert few(1, 1, 64) == 384 and few(1 << 20, 8, 128) == 16


def test_refusals(few):
    from kv_cache_quantization_hc_gb300 import hc
    assert few(0, 1, 64) == few(1, 0, 64) == few(1, 1, 0) == hc.HC_ERR_INVALID_ARG
    assert few(1, 1, 96) == few(1, 1, 256) == hc.HC_ERR_UNSUPPORTED
