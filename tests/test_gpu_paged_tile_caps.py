"""Attention over pages in tiles, capped scores: caps and factors whose
polynomial has terms that fp32 does not hold."""
import numpy as np
import pytest

from tests.paged_cases import Pages
from tests.test_gpu_serve import serve, workspace  # noqa: F401
from tests.test_gpu_serve_paged import check_attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("softcap,scale", [(3e5, 3e8), (6.9e5, 6.89e8), (2.4e5, 2.39e8), (1e5, 1e8), (6.9e5, 6.9e5)])
def test_caps_beside_the_largest_numbers(serve, workspace, dtype, d, sign, softcap, scale):  # noqa: F811
    """scale * (scale / softcap)^10 below and above fp32's end; scores of 0 and of a few units, some keys hidden in some
    tiles."""
    c = Pages(40, [300], [70], Hq=16, H=1, d=d, B=16, dtype=dtype, softcap=softcap, outliers=False, spread=1e-3,
              q_scale=1e3 / scale)
    c.q[::3] = 0
    assert min(c.new) * c.Hq // c.H > serve.attend_paged_few_rows(len(c.kv), c.H, c.d, c.table.shape[1] * c.B)
    check_attend(serve, workspace, c, scale=float(np.float32(sign * scale)))
