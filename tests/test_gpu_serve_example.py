"""The serving example: its steps agree with its cache, and with themselves when run again."""
import pytest

pytestmark = pytest.mark.gpu


def test_example_runs(capsys):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from examples import serve_int4
    # fp16 scores and probabilities' inputs (2^-11 each, scores of a few units), a bf16 output (2^-8)
    worst, tokens = serve_int4.main(4, 6)
    assert worst < 2.0 ** -8 + 16 * 2.0 ** -11
    again = serve_int4.main(4, 6)
    assert torch.equal(again[1], tokens) and tokens.shape == (4, 7)
    assert "requests" in capsys.readouterr().out
