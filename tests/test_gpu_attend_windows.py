"""Attention with a sliding window: windows that start with a tile of 128 keys, and what lies before a window."""
import numpy as np
import pytest

from oracle import serve as oserve
from tests.serve_cases import Cache, lse_bar, out_bar
from tests.test_gpu_serve import _check_attend, serve, workspace  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,d,window", [(32, 64, 128), (32, 128, 256), (32, 64, 300), (48, 64, 256), (48, 64, 300),
                                         (64, 64, 256), (64, 64, 512)])
def test_many_heads_to_a_key_head(serve, workspace, Hq, d, window):  # noqa: F811
    """A warp of 32 rows holds one token (or part of one), so no row of it sees a key of the tile before."""
    n = window + 480
    _check_attend(serve, workspace, Cache(41, [n], [n], Hq=Hq, H=1, d=d, B=16, group=32, window=window, outliers=False))


@pytest.mark.parametrize("window", [128, 256])
@pytest.mark.parametrize("at", [127, 255])
@pytest.mark.parametrize("Hq,H,scale", [(8, 2, "f16"), (8, 1, "f32")])
def test_a_key_before_the_window_dominates(serve, workspace, Hq, H, scale, at, window):  # noqa: F811
    """The other rows of the warp see key `at`, which outweighs what follows by 2^70 and more; the last token's window
    starts after it.  Rows that see the key keep nothing of the others (include/hc.h: below 2^-33 of the largest
    probability), which leaves the channels where its own value is zero out of the comparison for them."""
    import torch
    c = Cache(42, [700], [700], Hq=Hq, H=H, d=64, B=16, group=32, window=window, scale=scale)
    slot, row = c.table[0, at // 16], at % 16
    c.codes[slot, 0, :, row] = 0
    c.codes[slot, 0, :, row, 0] = 7
    c.scales[slot, 0, :, row] = oserve.round_like(60 / 7 if scale == "f32" else 8.5, scale)
    c.q[:, :, 0] = 8.0
    t, err = c.tensors(), torch.zeros(1, dtype=torch.int32, device="cuda")
    got, lse = serve.attend_int4(t["q"], t["codes"], t["scales"], t["table"], t["q_starts"], t["kv"], 700, workspace, err,
                                 window=window, return_lse=True)
    out, want_lse, weight, reach = c.expected()
    kept = np.ones(out.shape, bool)
    empty = np.repeat(oserve.int4_unpack(c.codes[slot, 1, :, row]) == 0, Hq // H, axis=0)     # [Hq, d]
    kept[at:at + window] = ~empty
    off = np.abs(got.double().cpu().numpy() - out) / out_bar(out, weight, reach, c.dtype).clip(1e-300)
    assert int(err) == 0 and off[kept].max() <= 1, off[kept].max()
    off = np.abs(lse.double().cpu().numpy() - want_lse) / lse_bar(want_lse, reach)
    assert off.max() <= 1, off.max()


@pytest.mark.parametrize("scale", ["f16", "f32"])
@pytest.mark.parametrize("d,group", [(64, 64), (128, 32), (128, 128)])
@pytest.mark.parametrize("new,Hq", [(1, 4), (3, 8), (30, 2), (300, 4)])
def test_rows_before_the_window_hold_anything(serve, workspace, new, Hq, d, group, scale):  # noqa: F811
    """Infinite and NaN scales in the rows that have left the window, in blocks that still hold visible ones."""
    c = Cache(43, [new + 461, 77 + new, new + 5], [new] * 3, Hq=Hq, H=2, d=d, B=32, group=group, scale=scale, window=70)
    r = np.random.default_rng(1)
    for i, n in enumerate(c.kv):
        first = max(0, n - c.new[i] - c.window + 1)
        for j in range(first // 32 * 32, first):
            c.scales[c.table[i, j // 32], :, :, j % 32] = r.choice([np.nan, np.inf, -np.inf, 6e4])
    _check_attend(serve, workspace, c)
