"""What the calls that serve from the paged buffer refuse, answered on the host
before any CUDA call (fake addresses and fake tensors, never dereferenced; CPU
only)."""
import ctypes
import math

import pytest

from tests.test_serve_devices import serve  # noqa: F401
from tests.test_serve_refusals import ROPES, A, _rope, _rows, hc  # noqa: F401


def _desc(hc, **kw):  # noqa: F811
    d = hc.hc_paged_desc(1, 2, 128, 16, 8, hc.HC_F16, 16 * 2 * 128, 0)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


DESCS = [(dict(n_layers=0), -1), (dict(n_layers=2), -1), (dict(n_kv_heads=0), -1), (dict(num_slots=0), -1), (dict(dtype=9), -1),
         (dict(d_head=96), -2), (dict(d_head=256), -2), (dict(block_size=8), -2), (dict(block_size=48), -2),
         (dict(slot_stride=16 * 2 * 128 - 8), -1), (dict(slot_stride=16 * 2 * 128 + 4), -1), (dict(slot_stride=1 << 40), -1)]


def _append(hc, q=None, k=None, v=None, q_out=None, n=8, heads=4, rope="none", token_rows=A, desc=None, kp=A, vp=2 * A, err=A):  # noqa: F811
    by = ctypes.byref
    return hc.lib().hc_append_paged(by(q or _rows(hc)), by(k or _rows(hc)), by(v or _rows(hc)), n, heads,
                                    None if rope == "none" else by(rope), token_rows, by(desc or _desc(hc)), kp, vp,
                                    by(q_out or _rows(hc)), err, None)


def _attend(hc, q=None, out=None, lse=None, n=8, heads=4, desc=None, kp=A, vp=A, tables=A, stride=20, width=20, starts=A,  # noqa: F811
            kv=A, n_req=2, max_new=4, ws=A, ws_bytes=None, err=A, scores="given", **how):
    by = ctypes.byref
    s = hc.hc_attend_scores(1, 0, 0.1, 0.0, None, None, None)
    for key, value in how.items():
        setattr(s, key, value)
    if ws_bytes is None:
        ws_bytes = hc.lib().hc_attend_paged_workspace()
    return hc.lib().hc_attend_paged(by(q or _rows(hc)), by(out or _rows(hc)), lse, n, heads, by(desc or _desc(hc)), kp, vp, tables,
                                    stride, width, starts, kv, n_req, max_new, by(s) if scores else None, ws, ws_bytes, err, None)


def _merge(hc, a=None, b=None, out=None, lse_a=A, lse_b=A, lse=A, dtype=None, n=8, heads=4, d=128):  # noqa: F811
    by = ctypes.byref
    return hc.lib().hc_merge_attention(by(a or _rows(hc)), lse_a, by(b or _rows(hc)), lse_b, by(out or _rows(hc)), lse,
                                       hc.HC_F16 if dtype is None else dtype, n, heads, d, None)


@pytest.mark.parametrize("kw,want", DESCS, ids=str)
def test_pages(hc, kw, want):  # noqa: F811
    assert _append(hc, desc=_desc(hc, **kw)) == want
    assert _attend(hc, desc=_desc(hc, **kw)) == want


def _bad_rows(hc):  # noqa: F811
    """NULL, not on 16 bytes, strides not on 16 bytes, a negative stride."""
    return (_rows(hc, None), _rows(hc, A + 8), _rows(hc, A, 1028), _rows(hc, A, 1024, 132), _rows(hc, A, -1024))


def test_append(hc):  # noqa: F811
    for kw in (dict(n=-1), dict(heads=-1), dict(token_rows=None), dict(token_rows=A + 4), dict(kp=None), dict(kp=A + 8),
               dict(vp=None), dict(vp=A + 8), dict(kp=A, vp=A), dict(err=None), dict(err=A + 2), dict(n=1 << 29, heads=6),
               dict(rope=_rope(hc, inverse=1)), dict(q_out=_rows(hc, A, 1024, 0)), dict(q_out=_rows(hc, A, 0, 128))):
        assert _append(hc, **kw) == hc.HC_ERR_INVALID_ARG, kw
    assert _append(hc, rope=_rope(hc, rot_dim=24)) == hc.HC_ERR_UNSUPPORTED
    for name in ("q", "k", "v", "q_out"):
        for r in _bad_rows(hc):
            assert _append(hc, **{name: r}) == hc.HC_ERR_INVALID_ARG, name


@pytest.mark.parametrize("kw", ROPES, ids=str)
def test_append_rotation(hc, kw):  # noqa: F811
    assert _append(hc, rope=_rope(hc, **kw)) == hc.HC_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(heads=0), dict(heads=3), dict(n_req=-1), dict(max_new=-1), dict(kp=None), dict(vp=A + 8), dict(tables=None),
    dict(tables=A + 1), dict(stride=19), dict(width=-1), dict(starts=None), dict(starts=A + 2), dict(kv=None), dict(kv=A + 1),
    dict(ws=None), dict(ws=A + 128), dict(ws_bytes=1000), dict(err=None), dict(lse=A + 2), dict(max_new=1 << 30),
    dict(n_req=1 << 22, width=1 << 16, stride=1 << 16), dict(n_req=1 << 20, max_new=1 << 28), dict(scores=None),
    dict(causal=2), dict(causal=-1), dict(window=-1), dict(causal=0, window=5), dict(causal=0, prefix_lens=A),
    dict(softmax_scale=math.inf), dict(softmax_scale=math.nan), dict(softcap=-1.0), dict(softcap=math.inf),
    dict(softcap=math.nan), dict(softcap=1e-45, softmax_scale=1.0), dict(softcap=3e38), dict(slopes=A + 2), dict(positions=A + 1),
    dict(prefix_lens=A + 2), dict(out=(A, 1024, 0)), dict(out=(A, 64, 128))], ids=str)
def test_attend(hc, kw):  # noqa: F811
    if "out" in kw:
        kw = dict(out=_rows(hc, *kw["out"]))
    assert _attend(hc, **kw) == hc.HC_ERR_INVALID_ARG


def test_attend_types_and_rows(hc):  # noqa: F811
    assert _attend(hc, desc=_desc(hc, dtype=hc.HC_F32)) == hc.HC_ERR_UNSUPPORTED
    for r in _bad_rows(hc):
        assert _attend(hc, q=r) == hc.HC_ERR_INVALID_ARG
        assert _attend(hc, out=r) == hc.HC_ERR_INVALID_ARG


def test_merge(hc):  # noqa: F811
    for kw in (dict(dtype=9), dict(n=-1), dict(heads=-1), dict(d=0), dict(lse_a=None), dict(lse_b=None), dict(lse_a=A + 2),
               dict(lse_b=A + 1), dict(lse=A + 2), dict(n=1 << 20, heads=1 << 10), dict(out=_rows(hc, A, 1024, 0))):
        assert _merge(hc, **kw) == hc.HC_ERR_INVALID_ARG, kw
    assert _merge(hc, d=96) == hc.HC_ERR_UNSUPPORTED
    for name in ("a", "b", "out"):
        for r in _bad_rows(hc):
            assert _merge(hc, **{name: r}) == hc.HC_ERR_INVALID_ARG, name


def test_nothing_to_do_launches_nothing(hc):  # noqa: F811
    none = _rows(hc, None, 0, 0)
    assert _append(hc, n=0, q=none, k=none, v=none, q_out=none, token_rows=None, rope=_rope(hc, positions=None)) == hc.HC_OK
    assert _attend(hc, n=0, q=none, out=none) == hc.HC_OK
    assert _attend(hc, n_req=0, kv=None, tables=None) == hc.HC_OK
    assert _attend(hc, max_new=0) == hc.HC_OK
    assert _merge(hc, n=0, a=none, b=none, out=none, lse_a=None, lse_b=None, lse=None) == hc.HC_OK
    assert _merge(hc, heads=0, a=none, b=none, out=none, lse_a=None, lse_b=None) == hc.HC_OK


def test_workspace_and_limit(hc):  # noqa: F811
    L = hc.lib()
    assert hc.lib().hc_attend_int4_workspace() <= L.hc_attend_paged_workspace() <= 32 << 20
    for bad in ((0, 8, 128, 100), (1, 0, 128, 100), (1, 8, 0, 100), (1, 8, 128, -1), (1, 8, 128, 1 << 31)):
        assert L.hc_attend_paged_few_rows(*bad) == hc.HC_ERR_INVALID_ARG
    assert L.hc_attend_paged_few_rows(1, 8, 96, 100) == hc.HC_ERR_UNSUPPORTED
    for keys in (0, 1, 1000, 100_000, (1 << 31) - 1):
        limits = [L.hc_attend_paged_few_rows(n, 8, 128, keys) for n in (1, 2, 8, 64, 1000, 1 << 20)]
        assert all(16 <= x <= 1024 and x % 16 == 0 for x in limits)


def _calls(make):
    """Arguments of a call of each kind, made by make(size, dtype)."""
    import torch
    n, Hq, H, d, B, S, R = 6, 4, 2, 64, 16, 9, 2
    i32, f32, f16 = torch.int32, torch.float32, torch.float16
    rows = lambda h: make((n, h, d), f16)
    pages = dict(k_pages=make((S, B, H, d), f16), v_pages=make((S, B, H, d), f16))
    err = make((1,), i32)
    return {
        "append_paged": dict(q=rows(Hq), k=rows(H), v=rows(H), token_rows=make((n,), torch.int64), err=err, q_out=rows(Hq),
                             positions=make((1, n), i32), table=make((50, d // 2, 2), f32), pair_axis=(0,) * (d // 2), **pages),
        "attend_paged": dict(q=rows(Hq), block_tables=make((R, 4), i32), q_starts=make((R + 1,), i32), kv_lens=make((R,), i32),
                             max_new=4, workspace=make((1 << 20,), torch.uint8), err=err, slopes=make((Hq,), f32),
                             positions=make((n,), i32), prefix_lens=make((R,), i32), out=rows(Hq), lse=make((n, Hq), f32),
                             return_lse=True, **pages),
        "merge_attention": dict(out_a=rows(Hq), lse_a=make((n, Hq), f32), out_b=rows(Hq), lse_b=make((n, Hq), f32), out=rows(Hq),
                                lse=make((n, Hq), f32))}


def _fake(device):
    import torch
    return lambda size, dtype: torch.empty(size, dtype=dtype, device=device)


@pytest.mark.parametrize("call", ["append_paged", "attend_paged", "merge_attention"])
def test_a_tensor_on_another_gpu_or_of_another_kind_is_refused(serve, call):  # noqa: F811
    import torch
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode(allow_non_fake_inputs=True):
        here, there, host = (_calls(_fake(d))[call] for d in ("cuda:0", "cuda:1", "cpu"))
        names = [k for k, v in here.items() if isinstance(v, torch.Tensor)]
        # the query's and the result's types and shapes are read with the GPU current, below with a GPU
        early = [k for k in names if k not in ("q", "q_out", "out")]
        changed = {k: [here[k].double(), here[k].bool()] for k in early}
        for k in early:
            if k not in ("table", "workspace"):      # of which a shorter one may do
                changed[k].append(here[k][:-1])
            if here[k].shape[-1] > 1:
                changed[k].append(torch.empty(*here[k].shape[:-1], 2 * here[k].shape[-1], dtype=here[k].dtype, device="cuda:0")[..., ::2])
    assert len(names) >= 6
    for name in names:
        for value in (there[name], host[name]):
            with pytest.raises(ValueError, match="cuda:[01]|CUDA tensor"):
                getattr(serve, call)(**{**here, name: value})
    for name in early:
        for value in changed[name]:
            with pytest.raises(ValueError):
                getattr(serve, call)(**{**here, name: value})


@pytest.mark.parametrize("call,name,value", [
    ("append_paged", "pairing", "pairs"), ("append_paged", "pair_axis", (1,) * 32), ("append_paged", "pair_axis", ()),
    ("attend_paged", "window", 1 << 31), ("attend_paged", "softcap", None),
    ("attend_paged", "softmax_scale", "x"), ("merge_attention", "out_a", None), ("attend_paged", "q", 3)])
def test_other_arguments(serve, call, name, value):  # noqa: F811
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode(allow_non_fake_inputs=True):
        here = _calls(_fake("cuda:0"))[call]
    with pytest.raises((ValueError, TypeError)):
        getattr(serve, call)(**{**here, name: value})
