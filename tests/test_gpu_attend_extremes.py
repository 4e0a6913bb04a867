"""Attention at the ends of its inputs' ranges, with rows for either kernel."""
import numpy as np  # noqa: F401
import pytest

from oracle import serve as oserve
from tests.serve_cases import Cache
from tests.test_gpu_serve import _check_attend, serve, workspace  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", ["f16", "f32"])
@pytest.mark.parametrize("mask", [dict(), dict(window=200), dict(causal=False)], ids=str)
@pytest.mark.parametrize("kv,new", [(450, 450), (130, 3), (1025, 500), (300, 450)])
def test_queries_of_zeros(serve, workspace, kv, new, mask, scale):  # noqa: F811
    """Every key counts alike; the last tile has runs of 32 keys that no row sees (and, at 300 keys, rows that see none)."""
    c = Cache(51, [kv], [new], Hq=4, H=4, d=64, B=16, group=32, scale=scale, **mask)
    c.q[::3] = 0
    c.q[-1] = 0
    _check_attend(serve, workspace, c)


@pytest.mark.parametrize("kv,new", [(450, 450), (130, 3)])
def test_keys_of_zeros(serve, workspace, kv, new):  # noqa: F811
    c = Cache(52, [kv], [new], Hq=4, H=4, d=128, B=16, group=128)
    for j in range(0, kv, 7):
        c.scales[c.table[0, j // 16], 0, :, j % 16] = 0
    for j in range(64, 96):
        c.scales[c.table[0, j // 16], 0, :, j % 16] = 0
    c.q[::5] = 0
    _check_attend(serve, workspace, c)


@pytest.mark.parametrize("mask", [dict(), dict(window=200), dict(causal=False)], ids=str)
@pytest.mark.parametrize("kv,new", [(450, 450), (130, 3), (1025, 500)])
def test_a_softmax_scale_of_zero(serve, workspace, kv, new, mask):  # noqa: F811
    _check_attend(serve, workspace, Cache(53, [kv], [new], Hq=4, H=4, d=64, B=16, group=32, **mask), softmax_scale=0.0)


@pytest.mark.parametrize("kv,new", [(450, 450), (130, 3)])
def test_a_negative_softmax_scale(serve, workspace, kv, new):  # noqa: F811
    _check_attend(serve, workspace, Cache(54, [kv], [new], Hq=4, H=4, d=64, B=16, group=32), softmax_scale=-0.2)


@pytest.mark.parametrize("large", [3e4, 1e8, 1e20])
@pytest.mark.parametrize("kv,new", [(1000, 450), (1000, 2)])
def test_keys_without_values_count(serve, workspace, kv, new, large):  # noqa: F811
    """Most keys have values of zeros and a small weight each, which the sum must not lose beside a few large values."""
    c = Cache(55, [kv], [new], Hq=1, H=1, d=64, B=16, group=32, scale="f32", outliers=False, hostile=False)
    c.codes[:, 0] = 0
    slot = c.table[0, 0]
    c.codes[slot, 0, :, 5, 0] = 7
    c.scales[:, 0] = oserve.round_like(0.943, "f32")            # key 5 scores 6.6, the others 0
    c.q[:, :, 0] = 8.0
    keep = c.scales[c.table[0, :2], 1].copy()
    c.scales[:, 1] = 0
    c.scales[c.table[0, :2], 1] = keep * large                    # keys 0 to 31
    c.scales = oserve.round_like(c.scales, "f32")
    _check_attend(serve, workspace, c)


@pytest.mark.parametrize("size", [1e30, 1e34, 3e37])
@pytest.mark.parametrize("kv,new", [(450, 450), (130, 3)])
def test_queries_near_the_largest_bf16(serve, workspace, kv, new, size):  # noqa: F811
    c = Cache(56, [kv], [new], Hq=4, H=4, d=64, B=16, group=32, q_scale=size, outliers=False)
    # scores up to 220; up to 7.4 where probabilities are fp16, which keep their bits down to 2^-22 of the largest
    for x in (3.0 if new == 3 else 0.1, 0.01):
        _check_attend(serve, workspace, c, softmax_scale=x / size)
