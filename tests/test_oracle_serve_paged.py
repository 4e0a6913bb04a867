"""The oracle of serving from the paged buffer, pinned to closed forms."""
import numpy as np
import pytest

from oracle import serve as oserve
from oracle import serve_paged as o
from tests.paged_cases import Pages

SHAPE = dict(Hq=4, H=2, d=16, B=8, dtype="f32")


def test_equal_scores_average_the_values():
    c = Pages(0, [11], [3], **SHAPE)
    c.q[:] = 0
    out, lse, *_ = c.expected()
    for t in range(3):
        j = np.arange(9 + t)
        v = c.v[c.table[0, j // 8], j % 8]
        assert np.allclose(out[t], v.mean(0).repeat(2, 0)) and np.allclose(lse[t], np.log(9 + t))


def test_agrees_with_the_4_bit_oracle():
    """The same keys and values, as codes with scales and as numbers."""
    r = np.random.default_rng(1)
    S, B, H, d = 4, 16, 2, 32
    codes = r.integers(0, 256, (S, 2, H, B, d // 2)).astype(np.uint8)
    scales = r.random((S, 2, H, B, 1))
    vals = oserve.values(codes, scales).transpose(1, 0, 3, 2, 4)
    q, table = r.standard_normal((9, 4, d)), np.array([[2, 0], [3, 1]])
    for kw in (dict(), dict(causal=False), dict(window=5)):
        a = oserve.attend(q, codes, scales, table, [0, 4, 9], [20, 31], B, **kw)
        b = o.attend(q, vals[0], vals[1], table, [0, 4, 9], [20, 31], **kw)
        assert all(np.allclose(x, y) for x, y in zip(a, b))


def test_masks_and_scores():
    c = Pages(2, [20, 13], [6, 13], **SHAPE)
    base = c.expected()[0]
    where = np.r_[14:20, 0:13]
    c.scores["positions"] = where
    assert np.array_equal(c.expected()[0], base)                          # the default positions
    c.scores.update(prefix_lens=[0, 0], softcap=1e9)
    assert np.allclose(c.expected()[0], base)
    c.scores.update(softcap=0.0, prefix_lens=[20, 99])
    whole = c.expected()[0]
    c.scores.update(prefix_lens=None, causal=False)
    assert np.array_equal(c.expected()[0], whole)                         # a prefix of everything: no mask
    c.scores.update(causal=True, slopes=np.full(4, 60.0))
    k = c.v[c.table[0, where[:6] // 8], where[:6] % 8].repeat(2, 1)
    assert np.allclose(c.expected()[0][:6], k)                            # a steep bias: a query sees itself
    c.scores.update(slopes=None, softcap=1e-6)
    c2 = Pages(2, [20, 13], [6, 13], **SHAPE)
    c2.q[:] = 0
    assert np.allclose(c.expected()[0], c2.expected()[0], atol=1e-4)      # a cap near 0: all keys alike
    c.scores.update(softcap=0.0, positions=np.full(19, -3))
    out, lse, *_ = c.expected()
    assert not out.any() and np.isneginf(lse).all()


@pytest.mark.parametrize("cut", [0, 7, 20])
def test_merge_of_parts_is_the_whole(cut):
    c = Pages(3, [20], [4], **SHAPE)
    whole, lse, *_ = c.expected()
    c.scores["prefix_lens"], c.scores["positions"] = [cut], np.full(4, -1)
    a, lse_a, *_ = c.expected()
    c.scores["prefix_lens"], c.scores["positions"] = None, np.arange(16, 20)
    parts = []
    for t in range(4):                                                    # keys cut.. of each query: a window
        c.scores["window"] = max(16 + t + 1 - cut, 0)
        if c.scores["window"]:
            x, y, *_ = c.expected()
            parts.append((x[t], y[t]))
        else:
            parts.append((np.full((4, 16), np.nan), np.full(4, -np.inf)))
    out, total = o.merge(a, lse_a, np.stack([x for x, _ in parts]), np.stack([y for _, y in parts]))
    if cut != 20:
        assert np.allclose(out, whole) and np.allclose(total, lse)
    else:
        assert np.array_equal(out, a) and np.array_equal(total, lse_a)


def test_merge_of_nothing():
    out, lse = o.merge(np.full((1, 1, 4), np.nan), np.full((1, 1), -np.inf), np.full((1, 1, 4), np.inf), np.full((1, 1), -np.inf))
    assert not out.any() and np.isneginf(lse).all()


def test_append_places_rows():
    r = np.random.default_rng(4)
    k, v, pages = r.standard_normal((3, 2, 16)), r.standard_normal((3, 2, 16)), np.zeros((2, 8, 2, 16))
    a, b = o.append(k, v, [9, -1, 0], pages, pages, "f32")
    assert np.array_equal(a[1, 1], k[0]) and np.array_equal(b[0, 0], v[2]) and np.count_nonzero(a) == 2 * 32
