"""The serving oracle against closed forms and a second route."""
import numpy as np
import pytest

from oracle import serve as oserve
from tests.serve_cases import Cache


def test_block_tables_by_hand():
    table = np.full((3, 3), -1, np.int32)
    table[0, :2] = [7, 9]
    table[2, 0] = 4
    got = oserve.block_tables([17, 0, 16], [1, 33, 1], [1, 2, 3, 5, 6], table, 16, 37)
    assert table.tolist() == [[7, 9, -1], [1, 2, 3], [4, 5, -1]]
    assert got["q_starts"].tolist() == [0, 1, 34, 35] and got["kv_lens"].tolist() == [18, 33, 17]
    assert got["token_rows"][0] == 9 * 16 + 1 and got["token_rows"][33] == 3 * 16 and got["token_rows"][34] == 5 * 16
    assert got["token_rows"][35] == -1 and got["token_req"][36] == -1 and got["n_taken"] == 4 and got["err"] == 0


def test_block_tables_shortage_and_bad_lengths():
    table = np.full((3, 2), -1, np.int32)
    got = oserve.block_tables([0, 40, 0], [20, 1, 3], [8], table, 16, 24)
    assert got["err"] == 8 | 16 and got["n_taken"] == 1
    assert got["kv_lens"].tolist() == [20, 0, 3]
    assert got["token_rows"].tolist() == list(range(128, 144)) + [-1] * 8


def test_rotation_turns_and_turns_back():
    r = np.random.default_rng(0)
    x = r.standard_normal((5, 2, 12)).astype(np.float32)
    pos = r.integers(0, 9, (2, 5))
    ang = np.arange(9)[:, None] * 0.7 ** np.arange(4)
    table = np.stack([np.cos(ang), np.sin(ang)], -1).astype(np.float32)
    for pairing in ("half_split", "interleaved"):
        y = oserve.rotate32(x, pos, table, (0, 1, 0, 1), pairing)
        assert np.array_equal(y[:, :, 8:], x[:, :, 8:])
        back = oserve.rotate32(y, pos, table, (0, 1, 0, 1), pairing, inverse=True)
        assert np.abs(back - x).max() < 1e-6
        lo, hi = ((1, 5) if pairing == "half_split" else (2, 3))
        a = ang[pos[1], 1][:, None]
        assert np.allclose(y[:, :, lo], x[:, :, lo] * np.cos(a) - x[:, :, hi] * np.sin(a), atol=1e-6)


def test_rotation_gradient_by_differences():
    """The inverse rotation of a cotangent is the gradient: differences of
    sum(w * rotate(x)), which is linear in x, so steps of 1 are exact up to rounding."""
    r = np.random.default_rng(1)
    x, w = (r.standard_normal((1, 1, 8)).astype(np.float32) for _ in range(2))
    ang = np.arange(4)[:, None] * np.ones(4)
    table = np.stack([np.cos(ang), np.sin(ang)], -1).astype(np.float32)
    f = lambda z: float((w.astype(np.float64) * oserve.rotate32(z, np.array([[3]]), table, (0,) * 4, "half_split")).sum())
    grad = oserve.rotate32(w, np.array([[3]]), table, (0,) * 4, "half_split", inverse=True)
    for c in range(8):
        e = np.zeros_like(x)
        e[0, 0, c] = 1
        assert abs((f(x + e) - f(x - e)) / 2 - grad[0, 0, c]) < 1e-5


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 5), (False, 0)])
def test_attention_against_a_dense_softmax(causal, window):
    """The paged loop against one dense masked softmax over gathered keys."""
    c = Cache(3, [9, 0, 33], [4, 2, 1], Hq=4, H=2, d=64, B=16, group=32, causal=causal, window=window)
    out, lse, _, _ = c.expected()
    vals = oserve.values(c.codes, np.nan_to_num(c.scales, posinf=0))
    for r in range(3):
        j = np.arange(c.kv[r])
        k = vals[np.maximum(c.table[r, j // 16], 0), 0, :, j % 16]
        v = vals[np.maximum(c.table[r, j // 16], 0), 1, :, j % 16]
        for i in range(c.new[r]):
            t, p = c.q_starts[r] + i, c.kv[r] - c.new[r] + i
            see = (j <= p if causal else j >= 0) & ((j > p - window) if window else True)
            for m in range(4):
                x = np.where(see, k[:, m // 2] @ c.q[t, m] / 8, -np.inf)
                if not see.any():
                    assert not out[t, m].any() and lse[t, m] == -np.inf
                    continue
                w = np.exp(x - np.logaddexp.reduce(x))
                assert np.allclose(out[t, m], w @ v[:, m // 2], rtol=1e-12, atol=1e-12)
                assert np.isclose(lse[t, m], np.logaddexp.reduce(x))
