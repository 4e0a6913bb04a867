"""Broadcast inputs of the serving calls, and outputs that would lie over one another."""
import pytest

from tests.test_gpu_serve import _err, serve, workspace  # noqa: F401

pytestmark = pytest.mark.gpu


def test_no_tokens_with_any_strides(serve, workspace):  # noqa: F811
    """A tensor without elements has strides that mean nothing."""
    import torch
    none = torch.empty(64, 4, 0, device="cuda").half().permute(2, 1, 0)          # [0, 4, 64]
    assert none.shape == (0, 4, 64) and none.stride(2) != 1
    codes, scales = serve.int4_cache(2, 2, 16, 64)
    err, kv = _err(), none[:, :2]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    pos, table, axes = i32([]), serve.rotation_table(4, 32, 1e4), (0,) * 32
    assert serve.rope_axes(none, pos, table, axes, err).shape == (0, 4, 64)
    assert serve.append_int4(none, kv, kv, torch.zeros(0, dtype=torch.int64, device="cuda"), codes, scales, pos, table, axes,
                             err).shape == (0, 4, 64)
    assert serve.attend_int4(none, codes, scales, i32([[0]]), i32([0, 0]), i32([3]), 1, workspace, err).shape == (0, 4, 64)


def test_broadcast_queries_and_outputs(serve, workspace):  # noqa: F811
    import torch
    n, Hq, H, d = 5, 4, 2, 64
    codes, scales = serve.int4_cache(4, H, 16, d)
    err = _err()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    table, axes = serve.rotation_table(n, d // 2, 1e4), (0,) * (d // 2)
    x = torch.randn(1, 1, d, device="cuda").half()
    wide, full = x.expand(n, Hq, d), x.expand(n, Hq, d).contiguous()
    a, b = (serve.rope_axes(t, pos, table, axes, err) for t in (wide, full))
    assert torch.equal(a, b)
    kv = torch.randn(n, H, d, device="cuda").half()
    rows = torch.arange(n, device="cuda")
    a, b = (serve.append_int4(t, kv, kv, rows, codes, scales, pos, table, axes, err) for t in (wide, full))
    assert torch.equal(a, b)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    tail = (codes, scales, i32([[0]]), i32([0, n]), i32([n]), n, workspace, err)
    a, b = (serve.attend_int4(t, *tail) for t in (wide, full))
    assert torch.equal(a, b) and int(err) == 0
    flat = torch.empty_like(x).expand(n, Hq, d)
    from kv_cache_quantization_hc_gb300 import hc
    for call in (lambda: serve.rope_axes(full, pos, table, axes, err, out=flat),
                 lambda: serve.append_int4(full, kv, kv, rows, codes, scales, pos, table, axes, err, q_out=flat),
                 lambda: serve.attend_int4(full, *tail, out=flat)):
        with pytest.raises(hc.HCError):
            call()
