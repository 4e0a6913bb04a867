"""The serving operators on the GPU against the oracle."""
import ctypes

import numpy as np
import pytest

from oracle import serve as oserve
from tests.serve_cases import DT, Cache, lse_bar, out_bar

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def serve():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from kv_cache_quantization_hc_gb300 import build
    build.build()
    from kv_cache_quantization_hc_gb300 import serve as s
    return s


@pytest.fixture(scope="module")
def workspace(serve):
    return serve.attend_workspace()


def _err():
    import torch
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------ block tables
def _tables_case(serve, cached, new, B, width, n_free, n_tokens, seed=0, pad=0):
    import torch
    r = np.random.default_rng(seed)
    n = len(cached)
    table = r.permutation(n * width).reshape(n, width).astype(np.int32)
    free = (n * width + r.permutation(n_free)).astype(np.int32)
    dev = torch.as_tensor(np.pad(table, ((0, 0), (0, pad)), constant_values=-7), device="cuda")[:, :width]
    i32 = lambda a: torch.as_tensor(np.asarray(a, np.int32), device="cuda")
    err = _err()
    got = serve.build_block_tables(i32(cached), i32(new), i32(free), dev, B, n_tokens, err)
    want = oserve.block_tables(cached, new, free, table, B, n_tokens)
    assert int(err) == want["err"]
    for name in ("q_starts", "kv_lens", "token_req", "token_pos", "token_rows"):
        assert np.array_equal(getattr(got, name).cpu().numpy(), want[name]), name
    assert int(got.n_taken) == want["n_taken"]
    assert np.array_equal(dev.cpu().numpy(), table)


@pytest.mark.parametrize("B", [16, 32, 64, 128])
@pytest.mark.parametrize("n_req", [1, 2, 63, 700])
def test_block_tables(serve, B, n_req):
    r = np.random.default_rng(n_req + B)
    cached, new = r.integers(0, 5 * B, n_req), r.integers(0, 3 * B, n_req)
    new[r.random(n_req) < 0.2] = 0
    _tables_case(serve, cached, new, B, 9, n_req * 5, int(new.sum()) + 3, seed=B, pad=n_req % 3)


def test_block_tables_many_requests(serve):
    """More requests than one pass over shared memory holds, empty ones among them."""
    r = np.random.default_rng(5)
    cached, new = r.integers(0, 40, 9001), r.integers(0, 4, 9001)
    new[4000:4200] = 0
    _tables_case(serve, cached, new, 16, 3, 9001, int(new.sum()))
    _tables_case(serve, cached, np.zeros(9001, int), 16, 3, 5, 2)


def test_block_tables_edges(serve):
    _tables_case(serve, [16], [1], 16, 2, 1, 1)                    # the first token of a block
    _tables_case(serve, [15], [1], 16, 1, 0, 1)                    # the last of one: no new block
    _tables_case(serve, [0, 0], [0, 0], 16, 1, 0, 0)               # nothing at all
    _tables_case(serve, [0, 5, 0], [40, 60, 20], 16, 5, 4, 120)    # free slots run out
    _tables_case(serve, [3, -1, 90, 2], [2, 3, 9, -4], 16, 6, 9, 14)  # bad lengths
    _tables_case(serve, [0, 7], [30, 30], 16, 4, 9, 41)            # more tokens than the arrays hold
    _tables_case(serve, [], [], 16, 1, 2, 3)                       # no request


# ------------------------------------------------------------------ rotation
def _rope_inputs(seed, n, axes, half, n_pos=97):
    r = np.random.default_rng(seed)
    pos = r.integers(0, n_pos, (axes, n)).astype(np.int32)
    ang = np.arange(n_pos)[:, None] * 100.0 ** (-np.arange(half) / half)
    table = np.stack([np.cos(ang), np.sin(ang)], -1).astype(np.float32)
    return r, pos, table, tuple(int(a) for a in r.integers(0, axes, half))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pairing", ["half_split", "interleaved"])
@pytest.mark.parametrize("n,H,d,rot,axes", [(1, 1, 64, 64, 1), (5, 3, 128, 96, 3), (33, 40, 128, 128, 3),
                                            (7, 2, 80, 20, 2), (300, 5, 64, 32, 4), (2, 1, 10, 6, 1),
                                            (3, 2, 256, 256, 8)])
def test_rope_axes_bit_exact(serve, dtype, pairing, n, H, d, rot, axes):
    import torch
    r, pos, table, pa = _rope_inputs(n + d, n, axes, rot // 2)
    x = oserve.round_like(r.standard_normal((n, H, d)) * 3, dtype)
    tt, pt, err = torch.as_tensor(table, device="cuda"), torch.as_tensor(pos, device="cuda"), _err()
    td = getattr(torch, DT[dtype])
    packed = torch.as_tensor(np.pad(x, ((0, 0), (1, 2), (0, 0))), device="cuda").to(td)
    for inverse in (False, True):
        want = oserve.round_like(oserve.rotate32(x, pos, table, pa, pairing, inverse), dtype)
        view = packed[:, 1:1 + H]
        got = serve.rope_axes(view, pt, tt, pa, err, pairing=pairing, inverse=inverse)
        assert np.array_equal(got.double().cpu().numpy(), want)
        # an output with gaps, off 16-byte alignment
        wide = torch.full((n, H, d + 1), -5.0, dtype=td, device="cuda")
        serve.rope_axes(view, pt, tt, pa, err, pairing=pairing, inverse=inverse, out=wide[:, :, 1:])
        assert np.array_equal(wide[:, :, 1:].double().cpu().numpy(), want) and bool((wide[:, :, 0] == -5).all())
        mine = view.clone()
        serve.rope_axes(mine, pt, tt, pa, err, pairing=pairing, inverse=inverse, out=mine)   # in place
        assert np.array_equal(mine.double().cpu().numpy(), want)
    assert int(err) == 0


def test_rope_axes_skips_positions_outside_the_table(serve):
    import torch
    _, pos, table, pa = _rope_inputs(0, 6, 2, 32)
    pa = (0, 1) * 16
    pos[1, 2], pos[0, 4] = -1, 97
    x = torch.randn(6, 3, 64, device="cuda")
    y, err = torch.full_like(x, 9.0), _err()
    serve.rope_axes(x, torch.as_tensor(pos, device="cuda"), torch.as_tensor(table, device="cuda"), pa, err, out=y)
    assert int(err) == 32
    assert bool((y[[2, 4]] == 9).all()) and not bool((y[[0, 1, 3, 5]] == 9).any())


def test_rope_table_is_the_frameworks(serve):
    t = serve.rotation_table(50, 32, 1e4).double().cpu().numpy()
    ang = np.arange(50)[:, None] * 1e4 ** (-np.arange(32) / 32)
    assert np.abs(t - np.stack([np.cos(ang), np.sin(ang)], -1)).max() < 1e-6


# -------------------------------------------------------------------- append
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d,H,Hq,B,group,scale,pairing,rot", [
    (128, 8, 32, 16, 32, "f16", "half_split", 128), (128, 1, 7, 64, 128, "f32", "interleaved", 96),
    (64, 3, 3, 32, 64, "f16", "half_split", 32), (64, 5, 0, 128, 32, "f32", "interleaved", 64),
    (128, 3, 6, 32, 64, "f16", "half_split", 0)])
@pytest.mark.parametrize("n", [1, 45])
def test_append_bit_exact(serve, dtype, d, H, Hq, B, group, scale, pairing, rot, n):
    import torch
    r, pos, table, pa = _rope_inputs(n + d + H, n, 3, max(rot // 2, 1))
    td = getattr(torch, DT[dtype])
    x = oserve.round_like(r.standard_normal((n, Hq + 2 * H, d)) * 2, dtype)
    x[:, :, 5] *= 8
    x[0, Hq] = 0                      # a row of zeros: scale 0
    x = oserve.round_like(x, dtype)
    S = 2 + -(-n // B)
    rows = r.permutation(S * B)[:n]
    rows[n // 2:n // 2 + (n > 1)] = -1  # a padding token
    codes = r.integers(0, 256, (S, 2, H, B, d // 2)).astype(np.uint8)
    scales = r.random((S, 2, H, B, d // group)).astype(np.float16).astype(np.float64)
    k32, v32 = x[:, Hq:Hq + H].astype(np.float32), x[:, Hq + H:].astype(np.float32)
    q32 = x[:, :Hq].astype(np.float32)
    if rot:
        k32, q32 = (oserve.rotate32(z, pos, table, pa, pairing) for z in (k32, q32))
    want_c, want_s = oserve.append(k32, v32, rows, codes, scales, B, group, scale)

    packed = torch.as_tensor(x, device="cuda").to(td)
    tc = torch.as_tensor(codes, device="cuda")
    ts = torch.as_tensor(scales, device="cuda").to(getattr(torch, DT[scale]))
    err = _err()
    q = serve.append_int4(packed[:, :Hq] if Hq else None, packed[:, Hq:Hq + H], packed[:, Hq + H:],
                          torch.as_tensor(rows, device="cuda"), tc, ts, torch.as_tensor(pos, device="cuda"),
                          torch.as_tensor(table, device="cuda") if rot else None, pa, err, pairing=pairing)
    assert int(err) == 0
    assert np.array_equal(tc.cpu().numpy(), want_c)
    assert np.array_equal(ts.double().cpu().numpy(), want_s)
    if Hq:
        assert np.array_equal(q.double().cpu().numpy(), oserve.round_like(q32, dtype))
    else:
        assert q is None


def test_append_equals_the_block_encoder(serve):
    """Unrotated tokens appended give the bytes that hc_encode_int4 gives for their blocks."""
    import torch
    from kv_cache_quantization_hc_gb300 import hc
    S, B, H, d = 5, 16, 4, 128
    pool = torch.randn(2, S, B, H, d, device="cuda").to(torch.bfloat16)
    wire_c, wire_s = serve.int4_cache(S, H, B, d)
    err = _err()
    order = torch.arange(S, dtype=torch.int32, device="cuda")
    hc.hc_encode_int4(pool[0], pool[1], hc.paged_desc(pool[0]), order, None, S, 32, hc.HC_F16, wire_c, wire_s, err)
    codes, scales = serve.int4_cache(S, H, B, d)
    serve.append_int4(None, pool[0].view(S * B, H, d), pool[1].view(S * B, H, d),
                      torch.arange(S * B, device="cuda"), codes, scales, None, None, None, err)
    assert int(err) == 0 and torch.equal(codes, wire_c) and torch.equal(scales, wire_s)


def test_append_refuses_rows_outside_the_cache(serve):
    import torch
    codes, scales = serve.int4_cache(2, 2, 16, 64)
    k = torch.ones(4, 2, 64, device="cuda")
    rows = torch.tensor([32, -2, 5, 1 << 40], device="cuda")
    q_out, err = torch.full_like(k, 3.0), _err()
    serve.append_int4(k, k, k, rows, codes, scales, None, None, None, err, q_out=q_out)
    assert int(err) == 1
    assert bool((q_out[[0, 1, 3]] == 3).all()) and bool((q_out[2] == 1).all())
    assert int(scales.count_nonzero()) == 2 * 2 * 2 and int(scales[0, :, :, 5].count_nonzero()) == 8


# ------------------------------------------------------------------ attention
def _check_attend(serve, workspace, c, **kw):
    import torch
    t, err = c.tensors(), _err()
    got, lse = serve.attend_int4(t["q"], t["codes"], t["scales"], t["table"], t["q_starts"], t["kv"],
                                 max(c.new + [0]), workspace, err, causal=c.causal, window=c.window,
                                 return_lse=True, **kw)
    out, want_lse, weight, reach = c.expected(kw.get("softmax_scale"))
    assert int(err) == 0
    g, gl = got.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(g).all()
    dead = np.isinf(want_lse)
    assert np.array_equal(np.isinf(gl), dead) and not g[dead].any()
    off = np.abs(g - out) / out_bar(out, weight, reach, c.dtype).clip(1e-300)
    assert off.max(initial=0) <= 1, off.max()
    off = np.abs(np.where(dead, 0, gl) - np.where(dead, 0, want_lse)) / lse_bar(want_lse, reach)
    assert off.max(initial=0) <= 1, off.max()
    return got, lse


SHAPES = [dict(Hq=32, H=8, d=128, B=16, group=32), dict(Hq=8, H=1, d=128, B=64, group=128),
          dict(Hq=14, H=2, d=64, B=32, group=64, scale="f32", dtype="f16"),
          dict(Hq=3, H=3, d=64, B=128, group=32, dtype="f16"), dict(Hq=10, H=2, d=128, B=32, group=64, scale="f32"),
          dict(Hq=5, H=1, d=128, B=16, group=32, scale="f32", dtype="f16"),
          dict(Hq=12, H=1, d=64, B=16, group=64, dtype="bf16")]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s.values())))
def test_attend_single_tokens(serve, workspace, shape):
    """One token per request, at the lengths around blocks and tiles; one request has none, one nothing cached."""
    kv = [1, 15, 16, 17, 31, 33, 127, 128, 129, 0, 255, 300, 513]
    _check_attend(serve, workspace, Cache(1, kv, [1] * 4 + [0] + [1] * 8, **shape))


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s.values())))
@pytest.mark.parametrize("mask", [dict(), dict(window=1), dict(window=40), dict(causal=False)], ids=str)
def test_attend_several_tokens(serve, workspace, shape, mask):
    """Drafts and chunks of prompts, with rows that see nothing (more queries than positions)."""
    _check_attend(serve, workspace, Cache(2, [5, 70, 33, 200, 3], [5, 3, 33, 7, 6], **shape, **mask))


@pytest.mark.parametrize("shape", SHAPES[:3] + SHAPES[4:5], ids=lambda s: "-".join(map(str, s.values())))
@pytest.mark.parametrize("mask", [dict(), dict(window=100), dict(causal=False)], ids=str)
def test_attend_prompts(serve, workspace, shape, mask):
    _check_attend(serve, workspace, Cache(3, [131, 1, 300, 260], [131, 1, 150, 2], **shape, **mask))


@pytest.mark.parametrize("n_req", [1, 3, 150])
def test_attend_split_over_ctas(serve, workspace, n_req):
    """One long request, few, and more requests than threads of a CTA: pieces
    held by several CTAs, CTAs that hold several pieces; the workspace is left as it was."""
    r = np.random.default_rng(n_req)
    kv = [6000] if n_req == 1 else [int(v) for v in r.integers(1, 900 if n_req < 100 else 300, n_req)]
    c = Cache(4, kv, [1] * n_req, Hq=8, H=2, d=64, B=16, group=32)
    a = _check_attend(serve, workspace, c)
    b = _check_attend(serve, workspace, c)
    assert all(bool((x == y).all()) for x, y in zip(a, b))        # the same bits every time
    assert int(workspace[:4096].count_nonzero()) == 0


@pytest.mark.parametrize("scale,spread", [("f32", 1e6), ("f32", 1e-12), ("f16", 1e-4), ("f16", 3e4), ("f32", 1.0)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("new", [1, 40])
def test_attend_ranges(serve, workspace, scale, spread, dtype, new):
    """Scales, queries and scores far from 1, and peaked softmaxes."""
    if dtype == "f16" and spread > 1e4:
        spread = 300.0                                            # the output has to hold the values
    c = Cache(5, [200, 77], [new, 1], Hq=4, H=1, d=64, B=16, group=32, scale=scale, dtype=dtype, spread=spread,
              outliers=False, q_scale=30.0 if dtype == "f16" else 1e5)
    for x in (3.0, 0.01):
        _check_attend(serve, workspace, c, softmax_scale=x / (spread * (30.0 if dtype == "f16" else 1e5)))


def test_attend_values_of_mixed_magnitude(serve, workspace):
    """Value scales that grow and shrink by orders of magnitude along the keys."""
    c = Cache(6, [700], [1], Hq=8, H=1, d=128, B=16, group=32, scale="f32")
    for j in range(700):
        c.scales[c.table[0, j // 16], 1, :, j % 16] *= 10.0 ** (j % 90 // 9 - 4)
    c.scales = oserve.round_like(c.scales, "f32")
    _check_attend(serve, workspace, c)


@pytest.mark.parametrize("new", [1, 50])
def test_attend_zero_values_and_queries(serve, workspace, new):
    c = Cache(7, [90, 60], [new, new], Hq=4, H=2, d=64, B=16, group=64, hostile=False)
    c.scales[:, 1] = 0
    c.q[0] = 0
    got, _ = _check_attend(serve, workspace, c)
    assert not bool(got.any())


@pytest.mark.parametrize("new", [1, 70])
def test_attend_strided_rows(serve, workspace, new):
    """Queries out of a packed buffer, outputs into one; other rows untouched."""
    import torch
    c = Cache(8, [100, 90], [new, new], Hq=8, H=2, d=64, B=32, group=32)
    t, err = c.tensors(), _err()
    n = t["q"].shape[0]
    packed = torch.randn(n, 12, 64, device="cuda").to(torch.bfloat16)
    packed[:, 2:10] = t["q"]
    wide = torch.full((n + 2, 11, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    a = serve.attend_int4(t["q"], t["codes"], t["scales"], t["table"], t["q_starts"], t["kv"], new, workspace, err)
    serve.attend_int4(packed[:, 2:10], t["codes"], t["scales"], t["table"], t["q_starts"], t["kv"], new, workspace,
                      err, out=wide[:n, 1:9])
    assert torch.equal(wide[:n, 1:9], a) and int(err) == 0
    assert bool((wide[:, 0] == 7).all()) and bool((wide[:, 9:] == 7).all()) and bool((wide[n:] == 7).all())


@pytest.mark.parametrize("new", [1, 40])
def test_attend_flags_bad_lengths_and_slots(serve, workspace, new):
    import torch
    c = Cache(9, [64, 50, 64], [new, new, new], Hq=4, H=1, d=64, B=16, group=32)
    t = c.tensors()
    out = torch.full_like(t["q"], 5.0)
    run = lambda err, kv=t["kv"], table=t["table"], max_new=new, starts=t["q_starts"]: serve.attend_int4(
        t["q"], t["codes"], t["scales"], table, starts, kv, max_new, workspace, err, out=out)
    good = run(_err()).clone()
    for bad in (-1, 10_000_000):
        kv = t["kv"].clone()
        kv[1] = bad
        out.fill_(5.0)
        err = _err()
        run(err, kv=kv)
        assert int(err) == 8
        assert bool((out[new:2 * new] == 5).all())
        assert torch.equal(out[:new], good[:new]) and torch.equal(out[2 * new:], good[2 * new:])
    starts = t["q_starts"].clone()
    starts[3] = 10_000                                             # past the queries
    out.fill_(5.0)
    err = _err()
    run(err, starts=starts, max_new=20_000)
    assert int(err) == 8 and bool((out[2 * new:] == 5).all()) and torch.equal(out[:2 * new], good[:2 * new])
    for slot in (-1, c.codes.shape[0]):
        table = t["table"].clone()
        table[0, 1] = slot
        err = _err()
        run(err, table=table)
        assert int(err) == 1 and torch.equal(out[new:], good[new:]) and bool(out.isfinite().all())


def test_attend_on_two_streams(serve):
    """Two streams at once, a workspace each, give what one after the other gives."""
    import torch
    c = [Cache(20 + i, [3000, 50 + i], [1, 3], Hq=8, H=2, d=128, B=16, group=32) for i in range(2)]
    t = [x.tensors() for x in c]
    ws = [serve.attend_workspace() for _ in c]
    err = _err()
    call = lambda i, s=None: serve.attend_int4(t[i]["q"], t[i]["codes"], t[i]["scales"], t[i]["table"],
                                               t[i]["q_starts"], t[i]["kv"], 3, ws[i], err, out=outs[i], stream=s)
    outs = [torch.empty_like(x["q"]) for x in t]
    for i in range(2):
        call(i)
    want = [o.clone() for o in outs]
    streams = [torch.cuda.Stream() for _ in c]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            call(i, s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want)) and int(err) == 0


def test_long_cache_offsets(serve, workspace):
    """A cache whose codes pass 4 GiB and whose rows' offsets pass 32 bits."""
    import torch
    S, H, B, d = 300_000, 8, 16, 128
    codes, scales = serve.int4_cache(S, H, B, d)
    slots = torch.tensor([[S - 1, 0, S - 2, 262_144, 131_073]], dtype=torch.int32, device="cuda")
    n = 70
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    k, v = (torch.randn(n, H, d, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(n, H, d, device="cuda", generator=g).to(torch.bfloat16)
    pos = torch.arange(n, device="cuda")
    rows = slots[0].long()[pos // B] * B + pos % B
    err = _err()
    serve.append_int4(None, k, v, rows, codes, scales, None, None, None, err)
    small_c, small_s = serve.int4_cache(5, H, B, d)
    serve.append_int4(None, k, v, pos, small_c, small_s, None, None, None, err)
    assert torch.equal(codes[slots[0].long()], small_c)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    order = i32([[0, 1, 2, 3, 4]])
    for m in (1, n):
        a = serve.attend_int4(q[:m], codes, scales, slots, i32([0, m]), i32([n]), m, workspace, err)
        b = serve.attend_int4(q[:m], small_c, small_s, order, i32([0, m]), i32([n]), m, workspace, err)
        assert torch.equal(a, b) and int(err) == 0


def test_step_in_a_graph(serve, workspace):
    """Block tables, append and attention captured once and replayed with new lengths."""
    import torch
    H, Hq, d, B, R = 2, 8, 64, 16, 3
    codes, scales = serve.int4_cache(64, H, B, d)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    cached, new = i32([0, 0, 0]), i32([1, 1, 1])
    free, tables, err = torch.arange(64, dtype=torch.int32, device="cuda"), torch.zeros(R, 8, dtype=torch.int32, device="cuda"), _err()
    table = serve.rotation_table(200, d // 2, 1e4)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    qkv = torch.randn(R, Hq + 2 * H, d, device="cuda", generator=g).to(torch.float16)

    def step():
        s = serve.build_block_tables(cached, new, free, tables, B, R, err)
        q = serve.append_int4(qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:], s.token_rows, codes, scales,
                              s.token_pos, table, (0,) * (d // 2), err)
        return serve.attend_int4(q, codes, scales, tables, s.q_starts, s.kv_lens, 1, workspace, err), s.n_taken

    step()
    torch.cuda.synchronize()
    codes.zero_(), scales.zero_(), tables.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, taken = step()
    codes2, scales2, tables2 = torch.zeros_like(codes), torch.zeros_like(scales), torch.zeros_like(tables)
    used = 0
    for it in range(20):
        cached.fill_(it)
        free.copy_(torch.arange(64, device="cuda").roll(-used))
        qkv.copy_(torch.randn(R, Hq + 2 * H, d, device="cuda", generator=g))
        graph.replay()
        used += int(taken)
        got = out.clone()
        keep = codes, scales, tables
        codes, scales, tables = codes2, scales2, tables2
        want, _ = step()
        codes, scales, tables = keep
        assert torch.equal(got, want) and torch.equal(codes, codes2) and torch.equal(tables, tables2)
    assert used == 6 and int(err) == 0
