"""Serving from the paged buffer on the GPU against the oracle."""
import numpy as np
import pytest

from oracle import serve as oserve
from oracle import serve_paged as opaged
from tests.paged_cases import DT, HALF, Pages, lse_bar, out_bar
from tests.test_gpu_serve import _rope_inputs, serve, workspace  # noqa: F401

pytestmark = pytest.mark.gpu


def _err():
    import torch
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# -------------------------------------------------------------------- append
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d,H,Hq,B,pairing,rot", [
    (128, 8, 32, 16, "half_split", 128), (128, 1, 7, 64, "interleaved", 96), (64, 3, 3, 32, "half_split", 32),
    (128, 5, 2, 16, "half_split", 96), (64, 5, 0, 128, "interleaved", 64), (128, 3, 6, 32, "half_split", 0)])
@pytest.mark.parametrize("n", [1, 45, 700])
def test_append_bit_exact(serve, dtype, d, H, Hq, B, pairing, rot, n):  # noqa: F811
    import torch
    r, pos, table, pa = _rope_inputs(n + d + H, n, 3, max(rot // 2, 1))
    td = getattr(torch, DT[dtype])
    x = oserve.round_like(r.standard_normal((n, Hq + 2 * H, d)) * 2, dtype)
    S = 2 + -(-n // B)
    rows = r.permutation(S * B)[:n]
    rows[n // 2:n // 2 + (n > 1)] = -1  # a padding token
    pages = oserve.round_like(r.standard_normal((2, S, B, H, d)), dtype)
    k, v, q = x[:, Hq:Hq + H], x[:, Hq + H:], x[:, :Hq]
    want_k, want_v = opaged.append(k, v, rows, pages[0], pages[1], dtype, pos, table if rot else None, pa, pairing)
    if rot:
        q = oserve.round_like(oserve.rotate32(q, pos, table, pa, pairing), dtype)
    packed = torch.as_tensor(x, device="cuda").to(td)
    # slots with gaps between them, as a layer of a buffer of several layers side by side
    wide = torch.full((2, S, 2, B, H, d), 5.0, dtype=td, device="cuda")
    wide[:, :, 0] = torch.as_tensor(pages, device="cuda").to(td)
    err = _err()
    got = serve.append_paged(packed[:, :Hq] if Hq else None, packed[:, Hq:Hq + H], packed[:, Hq + H:],
                             torch.as_tensor(rows, device="cuda"), wide[0, :, 0], wide[1, :, 0],
                             torch.as_tensor(pos, device="cuda"), torch.as_tensor(table, device="cuda") if rot else None, pa, err,
                             pairing=pairing)
    assert int(err) == 0
    assert np.array_equal(wide[0, :, 0].double().cpu().numpy(), want_k)
    assert np.array_equal(wide[1, :, 0].double().cpu().numpy(), want_v)
    assert bool((wide[:, :, 1] == 5).all())
    if Hq:
        assert np.array_equal(got.double().cpu().numpy(), q)
    else:
        assert got is None


def test_append_skips_bad_rows_and_positions(serve):  # noqa: F811
    import torch
    k_pages, v_pages = serve.paged_cache(2, 2, 16, 64, torch.float32)
    k = torch.ones(5, 2, 64, device="cuda")
    rows = torch.tensor([32, -2, 5, 1 << 40, 6], device="cuda")
    pos = torch.tensor([[1, 1, 1, 1, 99]], dtype=torch.int32, device="cuda")
    still = torch.zeros(10, 32, 2, device="cuda")
    still[..., 0] = 1
    for table, bits in ((None, 1), (still, 33)):
        k_pages.zero_(), v_pages.zero_()
        q_out, err = torch.full_like(k, 3.0), _err()
        serve.append_paged(k, k, k, rows, k_pages, v_pages, pos, table, (0,) * 32, err, q_out=q_out)
        assert int(err) == bits
        there = [2, 4] if table is None else [2]
        assert bool((q_out[there] == 1).all()) and bool((q_out[[i for i in range(5) if i not in there]] == 3).all())
        for pages in (k_pages, v_pages):
            assert int(pages.count_nonzero()) == len(there) * 128 and bool((pages[0, rows[there]] == 1).all())


# ----------------------------------------------------------------- attention
def check_attend(serve, workspace, c, scale=None, few=None, **kw):  # noqa: F811
    import torch
    t, err = c.tensors(), _err()
    few_rows = serve.attend_paged_few_rows(max(len(c.kv), 1), c.H, c.d, c.table.shape[1] * c.B)
    got, lse = serve.attend_paged(**t, max_new=max(c.new + [0]), workspace=workspace, err=err, softmax_scale=scale,
                                  return_lse=True, **kw)
    out, want_lse, weight, reach, far = c.expected(scale)
    assert int(err) == 0
    g, gl = got.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(g).all()
    dead = np.isinf(want_lse)
    assert np.array_equal(np.isinf(gl), dead) and not g[dead].any()
    rows = np.concatenate([np.full(n, n * c.Hq // c.H) for n in c.new]) if c.new else np.zeros(0)
    vmax = float(np.abs(c.v[np.isfinite(c.v)]).max(initial=0))
    cap = c.scores["softcap"]
    bars = [out_bar(out, weight, reach, far, vmax, c.d, c.dtype, f, cap) for f in (True, False)]
    bar = np.where((rows <= few_rows)[:, None, None], *bars).clip(1e-300)
    off = np.abs(g - out) / bar
    assert off.max(initial=0) <= 1, off.max()
    off = np.abs(np.where(dead, 0, gl) - np.where(dead, 0, want_lse)) / lse_bar(want_lse, reach, far, c.d, cap)
    assert off.max(initial=0) <= 1, off.max()
    return got, lse


SHAPES = [dict(Hq=32, H=8, d=128, B=16), dict(Hq=8, H=1, d=128, B=64, dtype="f16"), dict(Hq=14, H=2, d=64, B=32, dtype="f16"),
          dict(Hq=3, H=3, d=64, B=128), dict(Hq=10, H=2, d=128, B=32), dict(Hq=5, H=1, d=128, B=128, dtype="f16"),
          dict(Hq=12, H=1, d=64, B=16)]
IDS = dict(ids=lambda s: "-".join(map(str, s.values())) or "plain")
MODS = [dict(), dict(softcap=4.0), dict(slopes=True), dict(softcap=30.0, slopes=True)]


@pytest.mark.parametrize("shape", SHAPES, **IDS)
@pytest.mark.parametrize("mods", MODS, **IDS)
def test_attend_single_tokens(serve, workspace, shape, mods):  # noqa: F811
    """One token per request, at the lengths around blocks and tiles; one request has none, one nothing cached."""
    kv = [1, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 0, 255, 300, 513]
    check_attend(serve, workspace, Pages(1, kv, [1] * 4 + [0] + [1] * 11, **shape, **mods))


MASKS = [dict(), dict(window=1), dict(window=40), dict(causal=False), dict(prefix=[3, 500, -4, 70, 0]),
         dict(window=30, prefix=[5, 60, 0, 200, 2])]


@pytest.mark.parametrize("shape", SHAPES, **IDS)
@pytest.mark.parametrize("mask", MASKS, ids=str)
def test_attend_several_tokens(serve, workspace, shape, mask):  # noqa: F811
    """Drafts and chunks of prompts, with rows that see nothing (more queries than positions)."""
    check_attend(serve, workspace, Pages(2, [5, 70, 33, 200, 3], [5, 3, 33, 7, 6], **shape, **mask))


@pytest.mark.parametrize("shape", SHAPES[:4], **IDS)
@pytest.mark.parametrize("mask", [dict(), dict(window=100), dict(causal=False), dict(prefix=[40, 0, 280, 9])], ids=str)
@pytest.mark.parametrize("mods", MODS, **IDS)
def test_attend_prompts(serve, workspace, shape, mask, mods):  # noqa: F811
    check_attend(serve, workspace, Pages(3, [131, 1, 300, 260], [131, 1, 150, 2], **shape, **mask, **mods))


@pytest.mark.parametrize("shape", SHAPES, **IDS)
@pytest.mark.parametrize("share", [0.05, 0.6])
def test_attend_at_positions(serve, workspace, shape, share):  # noqa: F811
    """Some tokens of each request, computed again, with repeated, negative and too large positions among them."""
    r = np.random.default_rng(5)
    kv = [700, 40, 1, 250]
    pos = [np.sort(r.choice(n, max(1, int(n * share)), replace=False)) for n in kv]
    pos[1] = np.sort(np.concatenate([pos[1], [-7, -1, 5, 5, 40, 1000]]))
    for mods in (dict(), dict(window=60), dict(softcap=20.0, slopes=True), dict(prefix=[100, 0, 0, 250])):
        check_attend(serve, workspace, Pages(4, kv, [len(p) for p in pos], positions=np.concatenate(pos), **shape, **mods))


@pytest.mark.parametrize("n_req", [1, 3, 150])
def test_attend_split_over_ctas(serve, workspace, n_req):  # noqa: F811
    """One long request, few, and more requests than threads of a CTA: pieces held by several CTAs, CTAs
    that hold several pieces; the workspace is left as it was, and serves both caches."""
    import torch
    r = np.random.default_rng(n_req)
    kv = [6000] if n_req == 1 else [int(v) for v in r.integers(1, 900 if n_req < 100 else 300, n_req)]
    c = Pages(4, kv, [1] * n_req, Hq=8, H=2, d=64, B=16)
    a = check_attend(serve, workspace, c)
    b = check_attend(serve, workspace, c)
    assert all(torch.equal(x, y) for x, y in zip(a, b))        # the same bits every time
    assert int(workspace[:4096].count_nonzero()) == 0


SPLITS = [dict(kv_lens=[5000], new_lens=[80], Hq=12, H=1, d=64, B=16), dict(kv_lens=[4100, 3], new_lens=[300, 3], Hq=4, H=2, d=128, B=64, dtype="f16"),
          dict(kv_lens=[3000, 900, 2100], new_lens=[40, 700, 100], Hq=10, H=1, d=128, B=32),
          dict(kv_lens=[6000], new_lens=[450], Hq=2, H=2, d=64, B=128, window=2500), dict(kv_lens=[4000, 2600], new_lens=[200, 200], Hq=8, H=1, d=64, B=16, dtype="f16", softcap=20.0, slopes=True),
          dict(kv_lens=[3500], new_lens=[600], Hq=2, H=1, d=128, B=16, prefix=[3400], softcap=30.0)]


@pytest.mark.parametrize("case", SPLITS, ids=lambda c: "-".join(map(str, c["kv_lens"] + c["new_lens"])))
def test_attend_few_runs_of_many_keys(serve, workspace, case):  # noqa: F811
    """Fewer runs of 256 rows than SMs: their keys are shared out, and the parts joined."""
    import torch
    c = Pages(13, **case)
    assert max(c.new) * c.Hq // c.H > serve.attend_paged_few_rows(len(c.kv), c.H, c.d, c.table.shape[1] * c.B)
    a = check_attend(serve, workspace, c)
    b = check_attend(serve, workspace, c)
    assert all(torch.equal(x, y) for x, y in zip(a, b))        # the same bits every time
    assert int(workspace[:4096].count_nonzero()) == 0 and int(workspace[-256:].count_nonzero()) == 0


def test_attend_more_heads_than_places(serve, workspace):  # noqa: F811
    check_attend(serve, workspace, Pages(5, [50, 3], [1, 2], Hq=1200, H=1200, d=64, B=16))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("new", [1, 200])
def test_attend_ranges(serve, workspace, dtype, new):  # noqa: F811
    """Values far from 1, large scores and small ones, a negative scale."""
    for spread, q_scale in ((300.0, 30.0), (1e-4, 1.0)) + (((1e15, 1e6), (1e-12, 1e-8)) if dtype == "bf16" else ()):
        c = Pages(6, [200, 277], [1, new], Hq=4, H=1, d=64, B=16, dtype=dtype, spread=spread, q_scale=q_scale, outliers=False)
        for x in (3.0, 0.01, -1.0, 0.0):
            check_attend(serve, workspace, c, scale=x / (spread * q_scale))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("new", [1, 256])
@pytest.mark.parametrize("step", [0.05, -0.05])
def test_attend_scores_that_climb(serve, workspace, dtype, new, step):  # noqa: F811
    """Scores that rise (or fall) along the keys, so that the reference moves again and again."""
    c = Pages(7, [1500], [new], Hq=4, H=1, d=64, B=16, dtype=dtype, outliers=False)
    for j in range(1500):
        c.k[c.table[0, j // 16], j % 16] = oserve.round_like(step * j / 8, dtype)
    c.q[:] = 1.0
    check_attend(serve, workspace, c, scale=0.25)


@pytest.mark.parametrize("new", [1, 150])
def test_attend_zero_values_and_queries(serve, workspace, new):  # noqa: F811
    c = Pages(8, [290, 260], [new, new], Hq=4, H=2, d=64, B=16, hostile=False)
    c.v[:] = 0
    c.q[0] = 0
    got, _ = check_attend(serve, workspace, c)
    assert not bool(got.any())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("new", [1, 140])
def test_attend_values_beside_large_keys(serve, workspace, dtype, new):  # noqa: F811
    """Channels in which the keys with the largest scores hold zeros: what the others add has to be there."""
    c = Pages(9, [400], [new], Hq=4, H=1, d=64, B=32, dtype=dtype, outliers=False)
    for j in range(0, 400, 3):
        c.k[c.table[0, j // 32], j % 32] = oserve.round_like(c.k[c.table[0, j // 32], j % 32] * 3, dtype)
        c.v[c.table[0, j // 32], j % 32, :, 7:] = 0
    check_attend(serve, workspace, c, scale=0.5)


@pytest.mark.parametrize("new", [1, 170])
def test_attend_strided(serve, workspace, new):  # noqa: F811
    """Queries out of a packed buffer, outputs into one, pages of a buffer of several layers; the rest untouched."""
    import torch
    c = Pages(10, [200, 190], [new, new], Hq=8, H=2, d=64, B=32, hostile=False)
    t, err = c.tensors(), _err()
    a = serve.attend_paged(**t, max_new=new, workspace=workspace, err=err)
    n = t["q"].shape[0]
    packed = torch.randn(n, 12, 64, device="cuda").to(torch.bfloat16)
    packed[:, 2:10] = t["q"]
    S = t["k_pages"].shape[0]
    layers = torch.full((2, S, 3, 32, 2, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    layers[0, :, 1], layers[1, :, 1] = t["k_pages"], t["v_pages"]
    wide = torch.full((n + 2, 11, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    serve.attend_paged(**dict(t, q=packed[:, 2:10], k_pages=layers[0, :, 1], v_pages=layers[1, :, 1]), max_new=new,
                       workspace=workspace, err=err, out=wide[:n, 1:9])
    assert torch.equal(wide[:n, 1:9], a) and int(err) == 0
    assert bool((wide[:, 0] == 7).all()) and bool((wide[:, 9:] == 7).all()) and bool((wide[n:] == 7).all())
    # one query for all heads, the same pages for keys and values
    same = serve.attend_paged(**dict(t, q=t["q"][:, :1].expand(n, 8, 64), v_pages=t["k_pages"]), max_new=new,
                              workspace=workspace, err=err)
    want = serve.attend_paged(**dict(t, q=t["q"][:, :1].expand(n, 8, 64).contiguous(), v_pages=t["k_pages"].clone()), max_new=new,
                              workspace=workspace, err=err)
    assert torch.equal(same, want) and int(err) == 0


@pytest.mark.parametrize("new", [1, 140])
def test_attend_flags_bad_lengths_slots_and_positions(serve, workspace, new):  # noqa: F811
    import torch
    c = Pages(11, [164, 150, 164], [new, new, new], Hq=4, H=1, d=64, B=16)
    t = c.tensors()
    out = torch.full_like(t["q"], 5.0)

    def run(**kw):
        err = _err()
        serve.attend_paged(**dict(dict(t, max_new=new, workspace=workspace, err=err, out=out), **kw))
        return int(err)

    def same(a, b):  # up to a rounding: where keys are split depends on all of the call's lengths
        return bool(((a.float() - b.float()).abs() <= 2.0 ** -7 * b.float().abs() + 2.0 ** -14).all())

    assert run() == 0
    good = out.clone()
    for bad in (-1, 10_000_000):
        kv = t["kv_lens"].clone()
        kv[1] = bad
        out.fill_(5.0)
        assert run(kv_lens=kv) == 8
        assert bool((out[new:2 * new] == 5).all())
        assert same(out[:new], good[:new]) and same(out[2 * new:], good[2 * new:])
    starts = t["q_starts"].clone()
    starts[3] = 10_000                                             # past the queries
    out.fill_(5.0)
    assert run(q_starts=starts, max_new=20_000) == 8
    assert bool((out[2 * new:] == 5).all()) and same(out[:2 * new], good[:2 * new])
    for slot in (-1, c.k.shape[0]):
        table = t["block_tables"].clone()
        table[0, 1] = slot
        assert run(block_tables=table) == 1 and same(out[new:], good[new:]) and bool(out.isfinite().all())
    if new > 1:
        pos = torch.arange(3 * new, dtype=torch.int32, device="cuda") % new
        assert run(positions=pos) == 0
        want = out.clone()
        pos[5] = 100
        assert run(positions=pos) == 32 and same(out[new:], want[new:])


def test_padded_steps_and_nothing(serve, workspace):  # noqa: F811
    """Rows behind the last request, calls without tokens, requests or new tokens."""
    import torch
    for new in (1, 150):
        c = Pages(12, [190, 180], [new, new], Hq=4, H=1, d=64, B=16)
        t, err = c.tensors(), _err()
        want, want_lse = serve.attend_paged(**t, max_new=new, workspace=workspace, err=err, return_lse=True)
        q = torch.cat([t["q"], torch.full((5, 4, 64), float("nan"), device="cuda", dtype=torch.bfloat16)])
        out, lse = torch.full_like(q, 6.0), torch.full((2 * new + 5, 4), 6.0, device="cuda")
        serve.attend_paged(**dict(t, q=q), max_new=new, workspace=workspace, err=err, out=out, lse=lse, return_lse=True)
        assert torch.equal(out[:-5], want) and torch.equal(lse[:-5], want_lse) and bool((out[-5:] == 6).all())
        assert bool((lse[-5:] == 6).all()) and int(err) == 0
    empty = dict(t, q=t["q"][:0])
    assert serve.attend_paged(**empty, max_new=0, workspace=workspace, err=err).shape == (0, 4, 64)
    none = dict(t, block_tables=t["block_tables"][:0], kv_lens=t["kv_lens"][:0], q_starts=t["q_starts"][:1])
    out.fill_(2.0)
    serve.attend_paged(**dict(none, q=q), max_new=3, workspace=workspace, err=err, out=out)
    assert bool((out == 2).all()) and int(err) == 0


def test_long_pages_offsets(serve, workspace):  # noqa: F811
    """Pages whose elements pass 2^32."""
    import torch
    S, H, B, d = 300_000, 8, 16, 128
    k_pages, v_pages = serve.paged_cache(S, H, B, d)
    slots = torch.tensor([[S - 1, 0, S - 2, 262_144, 131_073]], dtype=torch.int32, device="cuda")
    n = 70
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    q, k, v = (torch.randn(n, H, d, device="cuda", generator=g).to(torch.bfloat16) for _ in range(3))
    pos = torch.arange(n, device="cuda")
    err = _err()
    serve.append_paged(None, k, v, slots[0].long()[pos // B] * B + pos % B, k_pages, v_pages, None, None, None, err)
    small = serve.paged_cache(5, H, B, d)
    serve.append_paged(None, k, v, pos, *small, None, None, None, err)
    assert torch.equal(k_pages[slots[0].long()], small[0]) and torch.equal(v_pages[slots[0].long()], small[1])
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    order = i32([[0, 1, 2, 3, 4]])
    for m, heads in ((1, 1), (n, 8)):
        wide = q[:m].repeat(1, heads, 1)
        a = serve.attend_paged(wide, k_pages, v_pages, slots, i32([0, m]), i32([n]), m, workspace, err)
        b = serve.attend_paged(wide, *small, order, i32([0, m]), i32([n]), m, workspace, err)
        assert torch.equal(a, b) and int(err) == 0


# --------------------------------------------------------------------- merge
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,Hq,d", [(1, 1, 64), (3, 5, 128), (700, 28, 128), (3001, 7, 64)])
def test_merge(serve, dtype, n, Hq, d):  # noqa: F811
    import torch
    r = np.random.default_rng(n)
    a, b = (oserve.round_like(r.standard_normal((n, Hq, d)) * 3, dtype) for _ in range(2))
    lse = [np.float32(r.standard_normal((n, Hq)) * 6).astype(np.float64) for _ in range(2)]
    lse[0][::3, 0], lse[1][::5, 0] = -np.inf, -np.inf
    a[::3, 0], b[::5, 0] = np.nan, np.inf                        # counts for nothing
    want, want_lse = opaged.merge(a, lse[0], b, lse[1])
    to = lambda x, dt: torch.as_tensor(x, device="cuda").to(dt)
    td = getattr(torch, DT[dtype])
    ta, tb, la, lb = to(a, td), to(b, td), to(lse[0], torch.float32), to(lse[1], torch.float32)
    out, total = serve.merge_attention(ta, la, tb, lb)
    # weights: a difference of log sums rounded at 2^-24 of at most 50, its exponential at 2^-21, the rest 2^-22
    bar = (50 * 2.0 ** -24 * 3 + 2.0 ** -20) * np.maximum(np.abs(np.nan_to_num(a, posinf=0)), np.abs(np.nan_to_num(b, posinf=0)))
    off = np.abs(out.double().cpu().numpy() - want) / (bar + HALF[dtype] * np.abs(want) * 1.01 + (2.0 ** -24 if dtype == "f16" else 1e-30))
    assert off.max() <= 1, off.max()
    gl = total.double().cpu().numpy()
    dead = np.isinf(want_lse)
    assert np.array_equal(np.isneginf(gl), dead)
    assert (np.abs(gl - want_lse)[~dead] <= 2.0 ** -22 * (2 + np.abs(want_lse[~dead]))).all()
    # in place, and into and out of packed buffers
    wide = torch.full((n, Hq + 3, d), 4.0, dtype=td, device="cuda")
    wide[:, 1:1 + Hq] = ta
    view, l2 = wide[:, 1:1 + Hq], la.clone()
    got = serve.merge_attention(view, l2, tb, lb, out=view, lse=l2)
    assert got[0] is view and torch.equal(view, out) and torch.equal(l2, total) and bool((wide[:, 1 + Hq:] == 4).all())


def test_merge_nothing(serve):  # noqa: F811
    import torch
    x, l = torch.zeros(0, 4, 64, device="cuda"), torch.zeros(0, 4, device="cuda")
    out, lse = serve.merge_attention(x, l, x, l)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
