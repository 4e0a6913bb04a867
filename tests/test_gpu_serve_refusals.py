"""What the Python calls of the serving operators refuse, and calls with nothing in them."""
import pytest

from tests.test_gpu_serve import serve, workspace  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture()
def args(serve, workspace):  # noqa: F811
    """Arguments of a call of each kind that is accepted."""
    import torch
    n, Hq, H, d, B, S = 6, 4, 2, 64, 16, 9
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    codes, scales = serve.int4_cache(S, H, B, d)
    rows = lambda h: torch.ones(n, h, d, dtype=torch.float16, device="cuda")
    err = i32([0])
    tables = i32([[0, 1, 2, -1], [3, 4, -1, -1]])
    pos, table = i32([list(range(n))]), serve.rotation_table(50, d // 2, 1e4)
    return {
        "build_block_tables": dict(cached_lens=i32([3, 20]), new_lens=i32([2, 4]), free_slots=i32([7, 8]),
                                   block_tables=tables, block_size=B, n_tokens=n, err=err),
        "rope_axes": dict(x=rows(Hq), positions=pos, table=table, pair_axis=(0,) * (d // 2), err=err),
        "append_int4": dict(q=rows(Hq), k=rows(H), v=rows(H), token_rows=torch.arange(n, device="cuda"), codes=codes,
                            scales=scales, positions=pos, table=table, pair_axis=(0,) * (d // 2), err=err),
        "attend_int4": dict(q=rows(Hq), codes=codes, scales=scales, block_tables=tables, q_starts=i32([0, 2, 6]),
                            kv_lens=i32([5, 24]), max_new=4, workspace=workspace, err=err)}


def _changes():
    cpu, half = (lambda t: t.cpu()), (lambda t: t.half())
    every_other = lambda t: t.repeat_interleave(2, -1)[..., ::2]
    return [
        ("build_block_tables", "cached_lens", cpu), ("build_block_tables", "cached_lens", lambda t: t.long()),
        ("build_block_tables", "new_lens", lambda t: t[:1]), ("build_block_tables", "free_slots", every_other),
        ("build_block_tables", "block_tables", lambda t: t[:1]), ("build_block_tables", "block_tables", every_other),
        ("build_block_tables", "n_tokens", lambda n: -1), ("build_block_tables", "n_tokens", lambda n: 1 << 40),
        ("build_block_tables", "out", lambda t: (1, 2)),
        ("rope_axes", "x", cpu), ("rope_axes", "x", lambda t: t.int()), ("rope_axes", "x", lambda t: t[0]),
        ("rope_axes", "x", every_other), ("rope_axes", "positions", lambda t: t[:, :3]),
        ("rope_axes", "positions", lambda t: t.long()), ("rope_axes", "table", half), ("rope_axes", "table", lambda t: t[:, :5]),
        ("rope_axes", "pair_axis", lambda a: (1,) * 32), ("rope_axes", "pair_axis", lambda a: ()),
        ("rope_axes", "pairing", lambda a: "pairs"), ("rope_axes", "err", half), ("rope_axes", "err", lambda t: t[:0]),
        ("rope_axes", "out", lambda a: a), ("rope_axes", "x", lambda t: None),
        ("append_int4", "k", lambda t: t[:, :1]), ("append_int4", "v", lambda t: t[:3]), ("append_int4", "v", lambda t: t.float()),
        ("append_int4", "q", lambda t: t[..., :32]), ("append_int4", "token_rows", lambda t: t.int()),
        ("append_int4", "token_rows", lambda t: t[:2]), ("append_int4", "codes", every_other),
        ("append_int4", "codes", lambda t: t[0]), ("append_int4", "scales", lambda t: t[:3]),
        ("append_int4", "scales", lambda t: t.double()), ("append_int4", "scales", every_other),
        ("attend_int4", "q", lambda t: t[..., :32]), ("attend_int4", "q", cpu), ("attend_int4", "codes", lambda t: t.char()),
        ("attend_int4", "block_tables", lambda t: t[:1]), ("attend_int4", "block_tables", lambda t: t.long()),
        ("attend_int4", "q_starts", lambda t: t[:2]), ("attend_int4", "kv_lens", half),
        ("attend_int4", "workspace", half), ("attend_int4", "lse", half), ("attend_int4", "max_new", lambda n: 1 << 33)]


@pytest.mark.parametrize("which", range(len(_changes())))
def test_refused_by_the_binding(serve, args, which):  # noqa: F811
    import torch
    call, name, change = _changes()[which]
    kw = dict(args[call])
    before = kw.get(name, torch.zeros(6, 4, device="cuda"))
    kw[name] = change(before)
    with pytest.raises(ValueError):
        getattr(serve, call)(**kw)


@pytest.mark.parametrize("call,name,change", [
    ("build_block_tables", "block_size", lambda b: 24), ("rope_axes", "pair_axis", lambda a: (0,) * 33),
    ("append_int4", "k", lambda t: __import__("torch").ones(6, 2, 68, device="cuda").half()[..., 2:66]),
    ("attend_int4", "q", lambda t: t.float()), ("attend_int4", "workspace", lambda t: t[:4096]),
    ("attend_int4", "workspace", lambda t: t[16:]), ("attend_int4", "window", lambda w: -1),
    ("attend_int4", "softmax_scale", lambda s: float("nan")), ("attend_int4", "q", lambda t: t[:, :3])],
    ids=lambda x: x if isinstance(x, str) else "")
def test_refused_by_the_library(serve, args, call, name, change):  # noqa: F811
    from kv_cache_quantization_hc_gb300 import hc
    kw = dict(args[call])
    kw[name] = change(kw.get(name))
    with pytest.raises((hc.HCError, ValueError)):
        getattr(serve, call)(**kw)


def test_wrong_kinds_of_argument(serve, args):  # noqa: F811
    for call, name, value in (("build_block_tables", "n_tokens", "6"), ("attend_int4", "max_new", 2.5),
                              ("attend_int4", "softmax_scale", "0.1"), ("rope_axes", "pair_axis", 3),
                              ("rope_axes", "stream", "0")):
        with pytest.raises((TypeError, AttributeError)):
            getattr(serve, call)(**{**args[call], name: value})


def test_accepted_as_they_are(serve, args):  # noqa: F811
    for call, kw in args.items():
        getattr(serve, call)(**kw)
    assert int(args["attend_int4"]["err"]) == 0


def test_nothing_in_a_call(serve, args):  # noqa: F811
    """No tokens, and no requests."""
    import torch
    a = args["rope_axes"]
    assert serve.rope_axes(a["x"][:0], a["positions"][:, :0], a["table"], a["pair_axis"], a["err"]).shape == (0, 4, 64)
    assert serve.rope_axes(a["x"][:, :0], a["positions"], a["table"], a["pair_axis"], a["err"]).shape == (6, 0, 64)
    a = args["append_int4"]
    q = serve.append_int4(a["q"][:0], a["k"][:0], a["v"][:0], a["token_rows"][:0], a["codes"], a["scales"],
                          a["positions"][:, :0], a["table"], a["pair_axis"], a["err"])
    assert q.shape == (0, 4, 64) and not bool(a["codes"].any())
    a = args["attend_int4"]
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    out, lse = serve.attend_int4(a["q"][:0], a["codes"], a["scales"], a["block_tables"], torch.zeros_like(a["q_starts"]),
                                 a["kv_lens"], 0, a["workspace"], a["err"], return_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    serve.attend_int4(a["q"][:0], a["codes"], a["scales"], a["block_tables"][:0], torch.zeros_like(a["q_starts"][:1]), none,
                      1, a["workspace"], a["err"])
    s = serve.build_block_tables(none, none, none, a["block_tables"][:0], 16, 3, a["err"])
    assert s.q_starts.tolist() == [0] and s.token_req.tolist() == [-1] * 3 and int(s.n_taken) == 0
    assert int(a["err"]) == 0
