"""The serving example's prompts, and the smoke test's, reach the prompt attention."""
import pytest

from tests.test_gpu_serve import serve  # noqa: F401

pytestmark = pytest.mark.gpu


def test_chunks_have_more_than_few_rows(serve):  # noqa: F811
    from examples import serve_int4 as e
    longest = e.GRID[0] * e.GRID[1] + 3 + 37 * 2                     # of three requests, as the smoke test has
    for n_req in (3, 5):
        assert min(longest, e.CHUNK) * (e.HQ // e.H) > serve.attend_few_rows(n_req, e.H, e.D)
    worst, tokens = e.main(3, 3, say=lambda line: None)
    assert worst < 2.0 ** -8 + 16 * 2.0 ** -11 and tokens.shape == (3, 4)
