"""The serving calls take tensors of one GPU only: a tensor on another is
refused before any CUDA call (fake tensors, which have shapes, types and
devices but no memory; CPU only)."""
import os
import shutil

import pytest


@pytest.fixture(scope="module")
def serve():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from kv_cache_quantization_hc_gb300 import build
    build.build()
    from kv_cache_quantization_hc_gb300 import serve
    return serve


def _args(make, serve):
    import torch
    n, Hq, H, d, B, S, R = 6, 4, 2, 64, 16, 9, 2
    i32, f16 = torch.int32, torch.float16
    rows = lambda h: make((n, h, d), f16)
    cache = dict(codes=make((S, 2, H, B, d // 2), torch.uint8), scales=make((S, 2, H, B, d // 32), f16))
    turn = dict(positions=make((1, n), i32), table=make((50, d // 2, 2), torch.float32), pair_axis=(0,) * (d // 2))
    err = make((1,), i32)
    return {
        "build_block_tables": dict(cached_lens=make((R,), i32), new_lens=make((R,), i32), free_slots=make((2,), i32),
                                   block_tables=make((R, 4), i32), block_size=B, n_tokens=n, err=err,
                                   out=serve.StepTables([make((k,), torch.int64 if i == 4 else i32)
                                                         for i, k in enumerate((R + 1, R, n, n, n, 1))])),
        "rope_axes": dict(x=rows(Hq), err=err, out=rows(Hq), **turn),
        "append_int4": dict(q=rows(Hq), k=rows(H), v=rows(H), token_rows=make((n,), torch.int64), err=err, q_out=rows(Hq),
                            **cache, **turn),
        "attend_int4": dict(q=rows(Hq), block_tables=make((R, 4), i32), q_starts=make((R + 1,), i32),
                            kv_lens=make((R,), i32), max_new=4, workspace=make((1 << 20,), torch.uint8), err=err,
                            out=rows(Hq), lse=make((n, Hq), torch.float32), **cache)}


@pytest.mark.parametrize("call", ["build_block_tables", "rope_axes", "append_int4", "attend_int4"])
def test_a_tensor_on_another_gpu_is_refused(serve, call):
    import torch
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode(allow_non_fake_inputs=True):
        here = _args(lambda size, dtype: torch.empty(size, dtype=dtype, device="cuda:0"), serve)[call]
        there = _args(lambda size, dtype: torch.empty(size, dtype=dtype, device="cuda:1"), serve)[call]
    names = [k for k, v in here.items() if isinstance(v, torch.Tensor)]
    assert len(names) >= 5
    for name in names:
        with pytest.raises(ValueError, match="cuda:[01]"):
            getattr(serve, call)(**{**here, name: there[name]})
    if call == "build_block_tables":
        for i in range(6):
            out = serve.StepTables([there["out"][j] if j == i else t for j, t in enumerate(here["out"])])
            with pytest.raises(ValueError, match="cuda:[01]"):
                serve.build_block_tables(**{**here, "out": out})
