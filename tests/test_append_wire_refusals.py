"""hc_append_int4_wire refuses what hc_append_int4 refuses (fake addresses, never dereferenced; CPU only)."""
import ctypes

from tests.test_serve_refusals import A, _cache, _rope, _rows, hc  # noqa: F401


def _append(hc, k=None, n=8, cache=None, codes=A, rope=None, err=A):  # noqa: F811
    by = ctypes.byref
    return hc.lib().hc_append_int4_wire(by(_rows(hc)), by(k or _rows(hc)), by(_rows(hc)), hc.HC_F16, n, 4,
                                        by(rope) if rope else None, A, by(cache or _cache(hc)), codes, A, by(_rows(hc)),
                                        err, None)


def test_refusals(hc):  # noqa: F811
    for kw in (dict(n=-1), dict(codes=None), dict(codes=A + 8), dict(err=None), dict(k=_rows(hc, A + 8)),
               dict(k=_rows(hc, None)), dict(rope=_rope(hc, inverse=1)), dict(cache=_cache(hc, scale_dtype=2))):
        assert _append(hc, **kw) == hc.HC_ERR_INVALID_ARG, kw
    assert _append(hc, cache=_cache(hc, d_head=96)) == hc.HC_ERR_UNSUPPORTED
    assert _append(hc, n=0) == hc.HC_OK
