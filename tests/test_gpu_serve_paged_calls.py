"""The calls that serve from the paged buffer as a program makes them: what the
binding refuses, streams, graphs, and a run of them together with the 4-bit cache."""
import numpy as np
import pytest

from tests.paged_cases import Pages
from tests.test_gpu_serve import serve, workspace  # noqa: F401
from tests.test_gpu_serve_streams import _owner

pytestmark = pytest.mark.gpu
CALLS = ["append_paged", "attend_paged", "merge_attention"]


@pytest.fixture()
def args(serve, workspace):  # noqa: F811
    """Arguments of a call of each kind that is accepted."""
    import torch
    n, Hq, H, d, B, S = 6, 4, 2, 64, 16, 9
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    rows = lambda h: torch.ones(n, h, d, dtype=torch.float16, device="cuda")
    k_pages, v_pages = serve.paged_cache(S, H, B, d, torch.float16)
    err, logs = i32([0]), torch.zeros(n, Hq, device="cuda")
    return {
        "append_paged": dict(q=rows(Hq), k=rows(H), v=rows(H), token_rows=torch.arange(n, device="cuda"), k_pages=k_pages,
                             v_pages=v_pages, positions=i32([list(range(n))]), table=serve.rotation_table(50, d // 2, 1e4),
                             pair_axis=(0,) * (d // 2), err=err),
        "attend_paged": dict(q=rows(Hq), k_pages=k_pages, v_pages=v_pages, block_tables=i32([[0, 1, 2, -1], [3, 4, -1, -1]]),
                             q_starts=i32([0, 2, 6]), kv_lens=i32([5, 24]), max_new=4, workspace=workspace, err=err),
        "merge_attention": dict(out_a=rows(Hq), lse_a=logs, out_b=rows(Hq), lse_b=logs + 1)}


def _changes():
    cpu, half = (lambda t: t.cpu()), (lambda t: t.half())
    every_other = lambda t: t.repeat_interleave(2, -1)[..., ::2]
    return [
        ("append_paged", "q", lambda t: t[:3]), ("append_paged", "q", lambda t: t.float()), ("append_paged", "q", every_other),
        ("append_paged", "k", lambda t: t[:, :1]), ("append_paged", "v", lambda t: t[:3]), ("append_paged", "k", cpu),
        ("append_paged", "q_out", lambda t: t.half()[:, :3]), ("append_paged", "q_out", lambda t: t),
        ("append_paged", "k_pages", lambda t: t[:, :, :1]), ("append_paged", "k_pages", lambda t: t[0]),
        ("append_paged", "v_pages", lambda t: t.bfloat16()), ("append_paged", "v_pages", lambda t: t.transpose(1, 2)),
        ("append_paged", "token_rows", lambda t: t.int()), ("append_paged", "table", lambda t: t[:, :5]),
        ("attend_paged", "q", lambda t: t[..., :32]), ("attend_paged", "q", lambda t: t.bfloat16()), ("attend_paged", "q", cpu),
        ("attend_paged", "out", lambda t: t), ("attend_paged", "out", lambda t: t.half()[:5]),
        ("attend_paged", "block_tables", lambda t: t[:1]), ("attend_paged", "block_tables", lambda t: t.long()),
        ("attend_paged", "q_starts", lambda t: t[:2]), ("attend_paged", "kv_lens", half), ("attend_paged", "workspace", half),
        ("attend_paged", "lse", half), ("attend_paged", "max_new", lambda n: 1 << 33), ("attend_paged", "slopes", half),
        ("attend_paged", "positions", lambda t: t), ("attend_paged", "prefix_lens", lambda t: t),
        ("merge_attention", "out_b", lambda t: t[:5]), ("merge_attention", "out_b", lambda t: t.float()),
        ("merge_attention", "lse_a", half), ("merge_attention", "lse_b", lambda t: t[:2]), ("merge_attention", "out", lambda t: t),
        ("merge_attention", "lse", half), ("merge_attention", "out_a", lambda t: t[0])]


@pytest.mark.parametrize("which", range(len(_changes())))
def test_refused_by_the_binding(serve, args, which):  # noqa: F811
    import torch
    call, name, change = _changes()[which]
    kw = dict(args[call])
    kw[name] = change(kw.get(name, torch.zeros(6, 4, 64, device="cuda")))
    with pytest.raises(ValueError):
        getattr(serve, call)(**kw)


@pytest.mark.parametrize("call,name,change", [
    ("append_paged", "v_pages", lambda t: "k_pages"), ("attend_paged", "workspace", lambda t: t[:4096]),
    ("attend_paged", "workspace", lambda t: t[16:]), ("attend_paged", "window", lambda w: -1),
    ("attend_paged", "softmax_scale", lambda s: float("nan")), ("attend_paged", "softcap", lambda s: -1.0),
    ("attend_paged", "q", lambda t: t[:, :3]), ("attend_paged", "window", lambda w: 4)],
    ids=lambda x: x if isinstance(x, str) else "")
def test_refused_by_the_library(serve, args, call, name, change):  # noqa: F811
    from kv_cache_quantization_hc_gb300 import hc
    kw = dict(args[call])
    value = change(kw.get(name))
    kw[name] = kw[value] if isinstance(value, str) else value
    if name == "window":
        kw["causal"] = value < 0
    with pytest.raises(hc.HCError):
        getattr(serve, call)(**kw)


def _made(result):
    return list(result) if isinstance(result, tuple) else [result]


@pytest.mark.parametrize("call", CALLS)
def test_outputs_are_allocated_on_the_calls_stream(serve, args, call):  # noqa: F811
    import torch
    kw = dict(args[call], **(dict(return_lse=True) if call == "attend_paged" else {}))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = [t.clone() for t in _made(getattr(serve, call)(**kw))]
    torch.cuda.synchronize()
    for stream, owner in ((side, side.cuda_stream), (side.cuda_stream, side.cuda_stream), (0, 0), (None, 0)):
        got = _made(getattr(serve, call)(**kw, stream=stream))
        torch.cuda.synchronize()
        assert all(_owner(t) == owner for t in got) and all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(side):
        got = _made(getattr(serve, call)(**kw))
    torch.cuda.synchronize()
    assert all(_owner(t) == side.cuda_stream for t in got)
    with pytest.raises(ValueError):              # cudaStreamPerThread
        getattr(serve, call)(**kw, stream=2)


def test_nothing_in_a_call(serve, args):  # noqa: F811
    a = args["append_paged"]
    kw = dict(a, q=a["q"][:0], k=a["k"][:0], v=a["v"][:0], token_rows=a["token_rows"][:0], positions=a["positions"][:, :0])
    assert serve.append_paged(**kw).shape == (0, 4, 64) and not bool(a["k_pages"].any())
    assert serve.append_paged(**dict(a, q=a["q"][:, :0])).shape == (6, 0, 64) and int(a["err"]) == 0


def test_two_streams_with_a_workspace_each(serve, workspace):  # noqa: F811
    """Calls of both kinds at the same time, many of them, each result that of the call by itself."""
    import torch
    cases = [Pages(20, [3000, 10, 700], [1, 1, 1], Hq=8, H=2, d=128, B=64),
             Pages(21, [1500, 600], [700, 90], Hq=4, H=2, d=64, B=16, dtype="f16", softcap=20.0)]
    calls, want = [], []
    for c, ws in zip(cases, (workspace, serve.attend_workspace())):
        calls.append(dict(c.tensors(), max_new=max(c.new), workspace=ws, err=torch.zeros(1, dtype=torch.int32, device="cuda")))
        want.append(serve.attend_paged(**calls[-1]))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(30):
        for i, s in enumerate(streams):
            got[i].append(serve.attend_paged(**calls[i], stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i]) and int(calls[i]["err"]) == 0


def test_two_graphs_share_a_workspace(serve, workspace):  # noqa: F811
    """A step of new tokens and one of a prompt, captured each, replayed in turn with other lengths, beside eager calls of
    the 4-bit cache over the same workspace."""
    import torch
    H, Hq, d, B = 2, 8, 64, 16
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    pages = [p.normal_(generator=g) for p in serve.paged_cache(48, H, B, d, torch.float16)]
    again = [p.clone() for p in pages]
    codes, scales = serve.int4_cache(48, H, B, d)
    codes.fill_(0x35), scales.fill_(0.01)
    turns, err = serve.rotation_table(400, d // 2, 1e4), i32([0])

    class Step:
        def __init__(self, n_req, tokens):
            self.max_new = tokens // n_req
            self.tables = (torch.arange(12 * n_req, device="cuda").view(n_req, 12) + (0 if n_req > 1 else 36)).int()
            self.qkv = torch.empty(tokens, Hq + 2 * H, d, device="cuda", dtype=torch.float16)
            self.starts, self.kv = i32([0] * (n_req + 1)), i32([0] * n_req)
            self.rows, self.at = torch.empty(tokens, dtype=torch.int64, device="cuda"), i32([[0] * tokens])

        def fill(self, cached, new):
            """New lengths, and new tokens; what no request has is padding."""
            self.qkv.normal_(generator=g)
            self.starts.copy_(i32([sum(new[:r]) for r in range(len(new) + 1)]))
            self.kv.copy_(i32([a + b for a, b in zip(cached, new)]))
            at = [(r, a + j) for r, (a, b) in enumerate(zip(cached, new)) for j in range(b)]
            rows = [int(self.tables[r, p // B]) * B + p % B for r, p in at]
            pad = self.rows.numel() - len(at)
            self.rows.copy_(torch.tensor(rows + [-1] * pad))
            self.at.copy_(i32([[p for _, p in at] + [0] * pad]))
            return len(at)

        def __call__(self, kv):
            x = self.qkv
            q = serve.append_paged(x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:], self.rows, *kv, self.at, turns, (0,) * (d // 2), err)
            return serve.attend_paged(q, *kv, self.tables, self.starts, self.kv, self.max_new, workspace, err, return_lse=True)

    steps = [Step(3, 3), Step(1, 160)]
    graphs = []
    for step in steps:
        step.fill([1] * step.kv.numel(), [step.max_new] * step.kv.numel())
        step(pages)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(pages)
        graphs.append((graph, out))
    for a, b in zip(pages, again):
        b.copy_(a)
    for it in range(12):
        used = [steps[0].fill([33 + it, 170 - it, it], [1, 1, 1]), steps[1].fill([2 * it], [160 - 13 * it])]
        for n, step, (graph, out) in zip(used, steps, graphs):
            graph.replay()
            got = [t.clone() for t in out]
            serve.attend_int4(steps[0].qkv[:, :Hq], codes, scales, steps[0].tables, i32([0, 1, 2, 3]), i32([30, 90, 1]), 1,
                              workspace, err)
            want = step(again)
            assert all(torch.equal(a[:n], b[:n]) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(pages, again))
    assert int(err) == 0


@pytest.mark.parametrize("new,dtype", [(1, "bf16"), (5, "f16"), (300, "bf16")])
def test_history_in_four_bits_and_pages(serve, workspace, new, dtype):  # noqa: F811
    """A request whose first blocks are in the 4-bit cache and the others in pages: both attended and joined, against one
    attention in float64 over all keys."""
    import torch
    from oracle import serve as oserve
    from oracle import serve_paged as opaged
    from tests.paged_cases import DT
    H, Hq, d, B, old, fresh = 2, 8, 64, 16, 13, 400
    r = np.random.default_rng(new)
    td = getattr(torch, DT[dtype])
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    err = i32([0])
    k, v = (oserve.round_like(r.standard_normal((old * B + fresh, H, d)), dtype) for _ in range(2))
    q = oserve.round_like(r.standard_normal((new, Hq, d)), dtype)
    to = lambda a: torch.as_tensor(np.ascontiguousarray(a), device="cuda").to(td)
    codes, scales = serve.int4_cache(old, H, B, d)
    serve.append_int4(None, to(k[:old * B]), to(v[:old * B]), torch.arange(old * B, device="cuda"), codes, scales, None, None,
                      None, err)
    held = -(-fresh // B)
    pages = serve.paged_cache(held, H, B, d, td)
    order = torch.as_tensor(r.permutation(held), device="cuda")
    at = torch.arange(fresh, device="cuda")
    serve.append_paged(None, to(k[old * B:]), to(v[old * B:]), order[at // B] * B + at % B, *pages, None, None, None, err)
    starts = i32([0, new])
    a = serve.attend_int4(to(q), codes, scales, torch.arange(old, dtype=torch.int32, device="cuda")[None], starts, i32([old * B]),
                          new, workspace, err, causal=False, return_lse=True)
    b = serve.attend_paged(to(q), *pages, order[None].int(), starts, i32([fresh]), new, workspace, err, return_lse=True)
    out, lse = serve.merge_attention(*a, *b)
    assert int(err) == 0
    hist = oserve.values(codes.cpu().numpy(), scales.double().cpu().numpy())     # [S, 2, H, B, d]
    both = []
    for i, x in enumerate((k, v)):
        first = np.moveaxis(np.asarray(hist, np.float64)[:, i], 1, 2).reshape(old * B, H, d)
        both.append(np.concatenate([first, x[old * B:], np.zeros((held * B - fresh, H, d))]).reshape(-1, B, H, d))
    want, want_lse, weight, _, _ = opaged.attend(q, *both, np.arange(old + held)[None], [0, new], [old * B + fresh])
    # each part's output and the joined one rounded (2^-8 or 2^-11 each), probabilities in the type, scores of up to a few
    # units from fp16 inputs of the 4-bit cache (2^-11 each way)
    half = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]
    assert (np.abs(out.double().cpu().numpy() - want) <= weight * (3 * half + 16 * 2.0 ** -11)).all()
    assert (np.abs(lse.double().cpu().numpy() - want_lse) <= 8 * 2.0 ** -11).all()


def test_example_runs(capsys):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from examples import reuse_chunks
    # the parts' bf16 outputs and the joined one (2^-8 each), probabilities in bf16 (2^-8), the 4-bit part's fp16 inputs
    bar = 3 * 2.0 ** -8 + 16 * 2.0 ** -11
    worst, tokens = reuse_chunks.main(3, 4)
    assert worst < bar
    again = reuse_chunks.main(3, 4)
    assert torch.equal(again[1], tokens) and tokens.shape == (3, 9)
    assert "requests" in capsys.readouterr().out
