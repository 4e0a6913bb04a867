"""What the serving calls refuse, answered on the host before any CUDA call
(fake addresses, never dereferenced; CPU only)."""
import ctypes
import os
import shutil

import pytest

A = 1 << 20   # an aligned fake address


@pytest.fixture(scope="module")
def hc():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from kv_cache_quantization_hc_gb300 import build, hc
    build.build()
    hc.lib()
    return hc


def _cache(hc, **kw):
    return hc.hc_int4_cache(*{**dict(n_kv_heads=2, d_head=128, block_size=16, num_slots=8, group=32,
                                     scale_dtype=hc.HC_F16), **kw}.values())


def _rows(hc, ptr=A, token=1024, head=128):
    return hc.hc_rows(ptr, token, head)


def _rope(hc, **kw):
    r = hc.hc_rope_axes_desc()
    for k, v in {**dict(positions=A, position_stride=64, table=A, n_axes=3, n_positions=100, rot_dim=128,
                        pairing=hc.HC_PAIR_HALF_SPLIT, inverse=0), **kw}.items():
        if k == "pair_axis":
            r.pair_axis[5] = v
        else:
            setattr(r, k, v)
    return r


CACHES = [(dict(n_kv_heads=0), "INVALID_ARG"), (dict(num_slots=0), "INVALID_ARG"), (dict(scale_dtype=2), "INVALID_ARG"),
          (dict(d_head=96), "UNSUPPORTED"), (dict(d_head=256), "UNSUPPORTED"), (dict(block_size=8), "UNSUPPORTED"),
          (dict(block_size=48), "UNSUPPORTED"), (dict(group=16), "UNSUPPORTED"), (dict(d_head=64, group=128), "UNSUPPORTED")]
ROPES = [dict(positions=None), dict(table=None), dict(table=A + 4), dict(n_axes=0), dict(n_axes=9), dict(n_positions=0),
         dict(rot_dim=0), dict(rot_dim=130), dict(rot_dim=15), dict(pairing=2), dict(inverse=2), dict(position_stride=3),
         dict(pair_axis=3)]


def _tables(hc, **kw):
    a = dict(cached=A, new=A, n_req=4, B=16, free=A, n_free=10, tables=A, stride=20, width=20, n_tokens=8, starts=A, kv=A,
             req=A, pos=A, rows=A, taken=A, err=A)
    a.update(kw)
    return hc.lib().hc_build_block_tables(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(n_req=-1), -1), (dict(n_free=-1), -1), (dict(n_tokens=-1), -1), (dict(B=0), -1), (dict(B=24), -2), (dict(B=256), -2),
    (dict(cached=None), -1), (dict(new=None), -1), (dict(free=None), -1), (dict(tables=None), -1), (dict(starts=None), -1),
    (dict(kv=None), -1), (dict(req=None), -1), (dict(pos=None), -1), (dict(rows=None), -1), (dict(taken=None), -1),
    (dict(err=None), -1), (dict(stride=19), -1), (dict(width=-1), -1), (dict(width=1 << 27, stride=1 << 27), -1),
    (dict(rows=A + 4), -1), (dict(kv=A + 2), -1)], ids=str)
def test_block_tables(hc, kw, want):
    assert _tables(hc, **kw) == want


def _axes(hc, dtype=None, n=8, heads=4, d=128, x=None, y=None, rope=None, err=A):
    return hc.lib().hc_rope_axes(ctypes.byref(x or _rows(hc)), ctypes.byref(y or _rows(hc)),
                                 hc.HC_BF16 if dtype is None else dtype, n, heads, d,
                                 ctypes.byref(rope or _rope(hc)), err, None)


@pytest.mark.parametrize("kw", [dict(dtype=7), dict(n=-1), dict(heads=-1), dict(d=1), dict(d=258), dict(err=None),
                                dict(err=A + 2), dict(n=1 << 30, heads=4)], ids=str)
def test_rope_axes(hc, kw):
    assert _axes(hc, **kw) == hc.HC_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", ROPES, ids=str)
def test_rotation_descriptors(hc, kw):
    assert _axes(hc, rope=_rope(hc, **kw)) == hc.HC_ERR_INVALID_ARG
    assert _append(hc, rope=_rope(hc, **kw)) == hc.HC_ERR_INVALID_ARG


def test_rope_axes_rows(hc):
    for r in (_rows(hc, None), _rows(hc, A + 1), _rows(hc, A, -1), _rows(hc, A, 1024, -8)):
        assert _axes(hc, x=r) == hc.HC_ERR_INVALID_ARG
        assert _axes(hc, y=r) == hc.HC_ERR_INVALID_ARG
    odd = _rope(hc, pairing=hc.HC_PAIR_INTERLEAVED, rot_dim=6)
    assert _axes(hc, d=9, rope=odd) == hc.HC_ERR_UNSUPPORTED


def _append(hc, q=None, k=None, v=None, q_out=None, dtype=None, n=8, heads=4, rope="none", token_rows=A, cache=None,
            codes=A, scales=A, err=A):
    by = ctypes.byref
    return hc.lib().hc_append_int4(by(q or _rows(hc)), by(k or _rows(hc)), by(v or _rows(hc)),
                                   hc.HC_F16 if dtype is None else dtype, n, heads,
                                   None if rope == "none" else by(rope), token_rows, by(cache or _cache(hc)), codes, scales,
                                   by(q_out or _rows(hc)), err, None)


def test_append(hc):
    for kw in (dict(dtype=9), dict(n=-1), dict(heads=-1), dict(token_rows=None), dict(token_rows=A + 4), dict(codes=None),
               dict(codes=A + 8), dict(scales=None), dict(scales=A + 8), dict(err=None), dict(n=1 << 29, heads=6),
               dict(rope=_rope(hc, inverse=1))):
        assert _append(hc, **kw) == hc.HC_ERR_INVALID_ARG, kw
    assert _append(hc, rope=_rope(hc, rot_dim=24)) == hc.HC_ERR_UNSUPPORTED
    for name in ("q", "k", "v", "q_out"):  # NULL, not on 16 bytes, strides not on 16 bytes
        for r in (_rows(hc, None), _rows(hc, A + 8), _rows(hc, A, 1028), _rows(hc, A, 1024, 132), _rows(hc, A, -1024)):
            assert _append(hc, **{name: r}) == hc.HC_ERR_INVALID_ARG, name


@pytest.mark.parametrize("kw,want", CACHES, ids=str)
def test_cache_shapes(hc, kw, want):
    want = getattr(hc, "HC_ERR_" + want)
    assert _append(hc, cache=_cache(hc, **kw)) == want
    assert _attend(hc, cache=_cache(hc, **kw)) == want


def _attend(hc, q=None, out=None, lse=None, dtype=None, n=8, heads=4, cache=None, codes=A, scales=A, tables=A, stride=20,
            width=20, starts=A, kv=A, n_req=2, max_new=4, causal=1, window=0, scale=0.1, ws=A, ws_bytes=None, err=A):
    by = ctypes.byref
    if ws_bytes is None:
        ws_bytes = hc.lib().hc_attend_int4_workspace()
    return hc.lib().hc_attend_int4(by(q or _rows(hc)), by(out or _rows(hc)), lse, hc.HC_F16 if dtype is None else dtype, n,
                                   heads, by(cache or _cache(hc)), codes, scales, tables, stride, width, starts, kv, n_req,
                                   max_new, causal, window, scale, ws, ws_bytes, err, None)


@pytest.mark.parametrize("kw", [
    dict(dtype=9), dict(n=-1), dict(heads=0), dict(heads=3), dict(n_req=-1), dict(max_new=-1), dict(codes=None),
    dict(scales=A + 4), dict(tables=None), dict(tables=A + 1), dict(stride=19), dict(width=-1), dict(starts=None),
    dict(starts=A + 2), dict(kv=None), dict(causal=2), dict(causal=-1), dict(window=-1), dict(causal=0, window=5),
    dict(scale=float("inf")), dict(scale=float("nan")), dict(ws=None), dict(ws=A + 128), dict(ws_bytes=1000), dict(err=None),
    dict(lse=A + 2), dict(max_new=1 << 30), dict(n_req=1 << 22, width=1 << 16, stride=1 << 16)], ids=str)
def test_attend(hc, kw):
    assert _attend(hc, **kw) == hc.HC_ERR_INVALID_ARG


def test_attend_types_and_rows(hc):
    assert _attend(hc, dtype=hc.HC_F32) == hc.HC_ERR_UNSUPPORTED
    for r in (_rows(hc, None), _rows(hc, A + 8), _rows(hc, A, 1028), _rows(hc, A, 1024, 132), _rows(hc, A, -1024)):
        assert _attend(hc, q=r) == hc.HC_ERR_INVALID_ARG
        assert _attend(hc, out=r) == hc.HC_ERR_INVALID_ARG


def test_nothing_to_do_launches_nothing(hc):
    """No tokens, no heads or no requests, with NULL where nothing is."""
    none = _rows(hc, None, 0, 0)
    assert _axes(hc, n=0, x=none, y=none, rope=_rope(hc, positions=None)) == hc.HC_OK
    assert _axes(hc, heads=0, x=none, y=none) == hc.HC_OK
    assert _append(hc, n=0, q=none, k=none, v=none, q_out=none, token_rows=None,
                   rope=_rope(hc, positions=None)) == hc.HC_OK
    assert _attend(hc, n=0, q=none, out=none) == hc.HC_OK
    assert _attend(hc, n_req=0, kv=None, tables=None) == hc.HC_OK
    assert _attend(hc, max_new=0) == hc.HC_OK


def test_workspace_size(hc):
    n = hc.lib().hc_attend_int4_workspace()
    assert 0 < n <= 32 << 20 and n == hc.lib().hc_attend_int4_workspace()
