"""Pages of float32 are written by append_paged and refused by attend_paged, which says so (fake tensors; CPU only)."""
import pytest

from tests.test_serve_devices import serve  # noqa: F401
from tests.test_serve_paged_refusals import _calls, _fake


def test_pages_of_float32_are_refused_by_name(serve):  # noqa: F811
    import torch
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode(allow_non_fake_inputs=True):
        here = _calls(_fake("cuda:0"))["attend_paged"]
        here = {k: here[k].float() if k in ("q", "k_pages", "v_pages", "out") else here[k] for k in here}
    assert here["k_pages"].dtype == torch.float32
    with pytest.raises(ValueError, match="attend_paged takes pages of float16 or bfloat16"):
        serve.attend_paged(**here)
