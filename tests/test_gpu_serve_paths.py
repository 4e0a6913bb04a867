"""Attention where the rule between its two kernels turns: many requests of a
few rows, which go to tiles of 256 rows, in one call with single tokens, which
do not; and the references that move."""
import numpy as np
import pytest

from tests.serve_cases import Cache
from tests.test_gpu_serve import _check_attend, serve, workspace  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mask", [dict(), dict(window=30), dict(causal=False)], ids=str)
@pytest.mark.parametrize("n_req,shape", [(40, dict(Hq=64, H=8, d=128, B=16, group=32)),
                                         (100, dict(Hq=10, H=2, d=64, B=32, group=64, scale="f32", dtype="f16")),
                                         (160, dict(Hq=9, H=1, d=128, B=64, group=128))],
                         ids=lambda x: str(x) if isinstance(x, int) else "-".join(map(str, x.values())))
def test_many_requests_of_few_rows(serve, workspace, n_req, shape, mask):  # noqa: F811
    """Lengths from 0 to 300 keys, 1 to 24 new tokens, some with rows that see nothing."""
    r = np.random.default_rng(n_req)
    kv = [int(v) for v in r.integers(0, 300, n_req)]
    new = [int(v) for v in r.integers(1, 25, n_req)]
    kv[:4], new[:4] = [1, 2, 150, 299], [24, 1, 1, 9]
    _check_attend(serve, workspace, Cache(31, kv, new, **shape, **mask))


@pytest.mark.parametrize("new", [1, 5, 120])
def test_scores_that_rise_along_the_keys(serve, workspace, new):  # noqa: F811
    """Each block of keys scores far above the ones before it: the reference has to follow."""
    c = Cache(32, [900, 333], [new, 1], Hq=8, H=2, d=64, B=16, group=32, scale="f32", outliers=False)
    for i, n in enumerate(c.kv):
        for j in range(n):
            c.scales[c.table[i, j // 16], 0, :, j % 16] *= 2.0 ** (j // 16 / 4)
    _check_attend(serve, workspace, c)


@pytest.mark.parametrize("new", [1, 9, 120])
def test_scores_that_fall_along_the_keys(serve, workspace, new):  # noqa: F811
    c = Cache(33, [900, 333], [new, 1], Hq=8, H=2, d=64, B=16, group=32, scale="f32", outliers=False)
    for i, n in enumerate(c.kv):
        for j in range(n):
            c.scales[c.table[i, j // 16], 0, :, j % 16] *= 2.0 ** (14 - j // 16 / 4)
    _check_attend(serve, workspace, c)


def test_more_requests_than_are_ordered(serve, workspace):  # noqa: F811
    """Above 256 requests the tiles' works are taken in the requests' order."""
    r = np.random.default_rng(3)
    kv = [int(v) for v in r.integers(0, 120, 300)]
    new = [int(v) for v in r.integers(0, 25, 300)]
    _check_attend(serve, workspace, Cache(34, kv, new, Hq=10, H=2, d=64, B=16, group=32))


@pytest.mark.parametrize("mask", [dict(), dict(window=600), dict(causal=False)], ids=str)
def test_prompts_over_caches_of_different_lengths(serve, workspace, mask):  # noqa: F811
    """Works of 1 to 21 tiles of keys, taken by the powers of two of what they see."""
    new = [300, 120, 64, 200, 1, 90]
    kv = [300, 2620, 764, 240, 1500, 50]
    _check_attend(serve, workspace, Cache(35, kv, new, Hq=8, H=1, d=64, B=32, group=64, dtype="f16", **mask))
