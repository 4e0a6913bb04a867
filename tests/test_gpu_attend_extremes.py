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
