"""Attention over pages in tiles with softmax_scale 0: every key counts alike, whatever its product."""
import numpy as np
import pytest

from oracle import serve as oserve
from tests.paged_cases import Pages
from tests.test_gpu_serve import serve, workspace  # noqa: F401
from tests.test_gpu_serve_paged import check_attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("mods", [dict(), dict(softcap=9.0), dict(slopes=True)], ids=str)
def test_no_scale(serve, workspace, d, new, mods):  # noqa: F811
    """Products of up to 2^126 times 0."""
    c = Pages(41, [300], [new], Hq=16, H=1, d=d, B=16, outliers=False, hostile=False, **mods)
    r = np.random.default_rng(42)
    c.q = oserve.round_like(c.q.clip(-4, 4) * 2.0 ** 57, "bf16")
    c.k = oserve.round_like(c.k.clip(-4, 4) * 2.0 ** 57, "bf16")
    c.k[r.random(c.k.shape[:3]) < 0.2] = 0
    check_attend(serve, workspace, c, scale=0.0)
