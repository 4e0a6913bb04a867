"""Output rows that lie over one another, as a broadcast tensor's do, are refused; broadcast inputs are not
(fake addresses, never dereferenced; CPU only)."""
import pytest

from tests.test_serve_refusals import _append, _attend, _axes, _rope, _rows, hc  # noqa: F401


@pytest.mark.parametrize("token,head", [(0, 128), (1024, 0), (0, 0), (120, 1024), (1024, 64)])
def test_outputs(hc, token, head):  # noqa: F811
    r = _rows(hc, token=token, head=head)
    assert _axes(hc, y=r) == hc.HC_ERR_INVALID_ARG
    assert _append(hc, q_out=r) == hc.HC_ERR_INVALID_ARG
    assert _attend(hc, out=r) == hc.HC_ERR_INVALID_ARG


def test_one_token_or_none(hc):  # noqa: F811
    """What is not used of the strides does not count."""
    flat = _rows(hc, token=0, head=0)
    assert _axes(hc, n=0, y=flat) == hc.HC_OK
    assert _append(hc, n=0, q_out=flat) == hc.HC_OK
    assert _attend(hc, n=0, out=flat) == hc.HC_OK
    assert _axes(hc, heads=0, y=flat) == hc.HC_OK
    # refused for its rope, after the rows have been looked at
    assert _axes(hc, n=1, heads=1, y=flat, rope=_rope(hc, n_axes=0)) == hc.HC_ERR_INVALID_ARG
