"""Attention over pages by the kernel of tiles of 256 rows: each of these calls
has only requests of more rows than go in pieces, which is asked of the rule, so
that a change of the rule cannot move them to the other kernel."""
import numpy as np
import pytest

from oracle import serve as oserve
from tests.paged_cases import Pages, lse_bar, out_bar
from tests.test_gpu_serve import serve, workspace  # noqa: F401
from tests.test_gpu_serve_paged import _err

pytestmark = pytest.mark.gpu
TYPES = pytest.mark.parametrize("d,dtype", [(64, "bf16"), (64, "f16"), (128, "bf16"), (128, "f16")])
MODS = [dict(), dict(softcap=4.0), dict(slopes=True), dict(softcap=30.0, slopes=True)]


def in_tiles(serve, c):  # noqa: F811
    """Whether every request goes to the tiles' kernel."""
    few = serve.attend_paged_few_rows(len(c.kv), c.H, c.d, c.table.shape[1] * c.B)
    return all(n * c.Hq // c.H > few for n in c.new)


def check(serve, workspace, c, scale=None, want_err=0):  # noqa: F811
    assert in_tiles(serve, c)
    err = _err()
    got, lse = serve.attend_paged(**c.tensors(), max_new=max(c.new), workspace=workspace, err=err, softmax_scale=scale,
                                  return_lse=True)
    assert int(err) == want_err
    out, want_lse, weight, reach, far = c.expected(scale)
    g, gl = got.double().cpu().numpy(), lse.double().cpu().numpy()
    dead = np.isinf(want_lse)
    assert np.isfinite(g).all() and np.array_equal(np.isneginf(gl), dead) and not g[dead].any()
    vmax = float(np.abs(c.v[np.isfinite(c.v)]).max(initial=0))
    cap = c.scores["softcap"]
    bar = out_bar(out, weight, reach, far, vmax, c.d, c.dtype, False, cap)
    if c.dtype == "f16":
        # out_bar's 2^-19 of the largest value is for 512 keys: a key's probability is off by 2^-25 at most where the row's
        # largest stands at 2^3 or more, so n keys by n * 2^-28
        keys = np.concatenate([np.full(n, float(kv)) for n, kv in zip(c.new, c.kv)])
        bar = bar + (keys[:, None, None] * 2.0 ** -28 - 2.0 ** -19) * vmax
    off = np.abs(g - out) / bar.clip(1e-300)
    assert off.max() <= 1, off.max()
    off = np.abs(np.where(dead, 0, gl) - np.where(dead, 0, want_lse)) / lse_bar(want_lse, reach, far, c.d, cap)
    assert off.max() <= 1, off.max()
    return got, lse


MASKS = [dict(), dict(window=1), dict(window=40), dict(causal=False), dict(prefix=[3, 500, -4, 300, 0]),
         dict(window=30, prefix=[5, 60, 0, 200, 2])]


@TYPES
@pytest.mark.parametrize("mods", MODS, ids=str)
@pytest.mark.parametrize("mask", MASKS, ids=str)
def test_masks(serve, workspace, d, dtype, mods, mask):  # noqa: F811
    """Rows that see nothing among them (more queries than keys)."""
    check(serve, workspace, Pages(50, [130, 70, 333, 200, 68], [70, 90, 66, 65, 68], Hq=16, H=1, d=d, B=16, dtype=dtype, **mask, **mods))


@pytest.mark.parametrize("shape", [dict(Hq=17, H=1, d=64, B=128), dict(Hq=17, H=1, d=128, B=32, dtype="f16"),
                                   dict(Hq=64, H=2, d=128, B=64), dict(Hq=128, H=1, d=64, B=32, dtype="f16"),
                                   dict(Hq=150, H=1, d=64, B=16)], ids=str)
@pytest.mark.parametrize("mods", MODS, ids=str)
def test_heads_and_blocks(serve, workspace, shape, mods):  # noqa: F811
    """Heads that divide a half of a tile's rows, whose queries come as boxes, and that do not."""
    check(serve, workspace, Pages(51, [131, 300, 65], [61, 150, 64], **shape, **mods))


@TYPES
def test_at_positions(serve, workspace, d, dtype):  # noqa: F811
    """Queries in between, with repeated, negative and too large positions among them."""
    r = np.random.default_rng(5)
    kv = [700, 140, 1, 250]
    pos = [np.sort(r.choice(n, m, replace=n < m)) for n, m in zip(kv, (90, 70, 66, 120))]
    pos[1] = np.sort(np.concatenate([pos[1], [-7, -1, 5, 5, 140, 1000]]))
    for mods in (dict(), dict(window=60), dict(softcap=20.0, slopes=True), dict(prefix=[100, 0, 0, 250])):
        check(serve, workspace, Pages(52, kv, [len(p) for p in pos], positions=np.concatenate(pos), Hq=16, H=1, d=d, B=16,
                                      dtype=dtype, **mods))


@TYPES
def test_ranges(serve, workspace, d, dtype):  # noqa: F811
    """Values far from 1, large scores and small ones, a negative scale and none."""
    for spread, q_scale in ((300.0, 30.0), (1e-4, 1.0)) + (((1e15, 1e6), (1e-12, 1e-8)) if dtype == "bf16" else ()):
        c = Pages(53, [200, 277], [70, 200], Hq=16, H=1, d=d, B=16, dtype=dtype, spread=spread, q_scale=q_scale, outliers=False)
        for x in (3.0, 0.01, -1.0, 0.0):
            check(serve, workspace, c, scale=x / (spread * q_scale))


@TYPES
@pytest.mark.parametrize("step", [0.05, -0.05])
@pytest.mark.parametrize("mods", MODS, ids=str)
def test_scores_that_climb(serve, workspace, d, dtype, step, mods):  # noqa: F811
    """Scores that rise (or fall) along the keys, so that the reference moves again and again."""
    c = Pages(54, [1500], [80], Hq=16, H=1, d=d, B=16, dtype=dtype, outliers=False, **mods)
    for j in range(1500):
        c.k[c.table[0, j // 16], j % 16] = oserve.round_like(step * j / 8, dtype)
    c.q[:] = 1.0
    check(serve, workspace, c, scale=0.25)


@TYPES
def test_one_row_climbs(serve, workspace, d, dtype):  # noqa: F811
    """One row of a warp whose reference moves at every tile, beside rows whose scores are level, with keys seen partly."""
    c = Pages(55, [1500], [80], Hq=16, H=1, d=d, B=16, dtype=dtype, outliers=False)
    for j in range(1500):
        c.k[c.table[0, j // 16], j % 16, :, 0] = oserve.round_like(-0.05 * j, dtype)
    c.q[..., 0] = 0
    c.q[5, 3], c.q[70] = 0, 0
    c.q[5, 3, 0], c.q[70, :, 0] = 8.0, np.arange(16) - 5
    check(serve, workspace, c, scale=0.25)


@TYPES
def test_zero_values_and_queries(serve, workspace, d, dtype):  # noqa: F811
    c = Pages(56, [290, 260], [90, 66], Hq=16, H=1, d=d, B=16, dtype=dtype, hostile=False)
    c.v[:] = 0
    c.q[0] = 0
    got, _ = check(serve, workspace, c)
    assert not bool(got.any())


@TYPES
def test_values_beside_large_keys(serve, workspace, d, dtype):  # noqa: F811
    """Channels in which the keys with the largest scores hold zeros: what the others add has to be there."""
    c = Pages(57, [400], [70], Hq=16, H=1, d=d, B=32, dtype=dtype, outliers=False)
    for j in range(0, 400, 3):
        c.k[c.table[0, j // 32], j % 32] = oserve.round_like(c.k[c.table[0, j // 32], j % 32] * 3, dtype)
        c.v[c.table[0, j // 32], j % 32, :, 7:] = 0
    check(serve, workspace, c, scale=0.5)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("softcap,x", [(1e-35, 1.0), (1e-20, 1.0), (1e-3, 0.3), (1.0, 300.0), (2e5, 1.0), (3e30, 1.0), (5.0, -2.0), (5.0, 0.0),
                                       (0.02, 900.0)])
def test_caps_far_from_one(serve, workspace, dtype, softcap, x):  # noqa: F811
    """Scores of about x times the cap, some keys hidden in each tile."""
    c = Pages(58, [200, 277], [66, 200], Hq=16, H=1, d=64, B=16, dtype=dtype, softcap=softcap, outliers=False)
    check(serve, workspace, c, scale=float(np.float32(x * softcap / 64)))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("mask", [dict(prefix=[20, 300]), dict(prefix=[20, 300], window=50)], ids=str)
@pytest.mark.parametrize("softcap", [0.0, 6.0])
def test_more_queries_than_keys_with_a_bias(serve, workspace, dtype, mask, softcap):  # noqa: F811
    """Positions below 0 see the prefix only, at a distance counted from -1."""
    check(serve, workspace, Pages(59, [30, 300], [75, 420], Hq=16, H=1, d=64, B=16, dtype=dtype, slopes=True, softcap=softcap, **mask))


@pytest.mark.parametrize("Hq", [32, 34])
def test_strided(serve, workspace, Hq):  # noqa: F811
    """Queries out of a packed buffer (by boxes and not), outputs into one, pages of a buffer of several layers; the rest
    untouched.  One query for all heads; the same pages for keys and values."""
    import torch
    c = Pages(60, [200, 190], [70, 90], Hq=Hq, H=2, d=64, B=32, hostile=False)
    assert in_tiles(serve, c)
    t, err = c.tensors(), _err()
    call = lambda **kw: serve.attend_paged(**dict(t, max_new=90, workspace=workspace, err=err, **kw))
    a, n = call(), 160
    packed = torch.randn(n, Hq + 4, 64, device="cuda").to(torch.bfloat16)
    packed[:, 2:2 + Hq] = t["q"]
    S = t["k_pages"].shape[0]
    layers = torch.full((2, S, 3, 32, 2, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    layers[0, :, 1], layers[1, :, 1] = t["k_pages"], t["v_pages"]
    for lead in (1, 3):                               # rows on 32-byte boundaries, whose channels are 128 bytes a head
        wide = torch.full((n + 2, Hq + 3, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        serve.attend_paged(**dict(t, q=packed[:, 2:2 + Hq], k_pages=layers[0, :, 1], v_pages=layers[1, :, 1]), max_new=90,
                           workspace=workspace, err=err, out=wide[:n, lead:lead + Hq])
        assert torch.equal(wide[:n, lead:lead + Hq], a) and bool((wide[:, :lead] == 7).all())
        assert bool((wide[:, lead + Hq:] == 7).all()) and bool((wide[n:] == 7).all())
    flat = torch.full((n * Hq * 64 + 8,), 7.0, dtype=torch.bfloat16, device="cuda")   # rows on 16-byte boundaries only
    call(out=flat[8:].view(n, Hq, 64))
    assert torch.equal(flat[8:].view(n, Hq, 64), a) and bool((flat[:8] == 7).all())
    one = t["q"][:, :1].expand(n, Hq, 64)
    same = serve.attend_paged(**dict(t, q=one, v_pages=t["k_pages"]), max_new=90, workspace=workspace, err=err)
    want = serve.attend_paged(**dict(t, q=one.contiguous(), v_pages=t["k_pages"].clone()), max_new=90, workspace=workspace, err=err)
    assert torch.equal(same, want)
    token = t["q"][:1].expand(n, Hq, 64)              # one token's queries for all
    same = serve.attend_paged(**dict(t, q=token), max_new=90, workspace=workspace, err=err)
    want = serve.attend_paged(**dict(t, q=token.contiguous()), max_new=90, workspace=workspace, err=err)
    assert torch.equal(same, want) and int(err) == 0


@TYPES
def test_flags_bad_lengths_slots_and_positions(serve, workspace, d, dtype):  # noqa: F811
    import torch
    new = 70
    c = Pages(61, [164, 150, 164], [new] * 3, Hq=16, H=1, d=d, B=16, dtype=dtype)
    assert in_tiles(serve, c)
    t = c.tensors()
    out = torch.full_like(t["q"], 5.0)

    def run(**kw):
        err = _err()
        serve.attend_paged(**dict(dict(t, max_new=new, workspace=workspace, err=err, out=out), **kw))
        return int(err)

    assert run() == 0
    good = out.clone()
    for bad in (-1, 10_000_000):
        kv = t["kv_lens"].clone()
        kv[1] = bad
        out.fill_(5.0)
        assert run(kv_lens=kv) == 8
        assert bool((out[new:2 * new] == 5).all())
        assert torch.equal(out[:new], good[:new]) and torch.equal(out[2 * new:], good[2 * new:])
    starts = t["q_starts"].clone()
    starts[3] = 10_000                                             # past the queries
    out.fill_(5.0)
    assert run(q_starts=starts, max_new=20_000) == 8
    assert bool((out[2 * new:] == 5).all()) and torch.equal(out[:2 * new], good[:2 * new])
    zeroed = c.k.copy(), c.v.copy()
    for slot in (-1, c.k.shape[0], 2 ** 31 - 1):                   # its block is taken as zeros
        table = t["block_tables"].clone()
        table[0, 1] = slot
        assert run(block_tables=table) == 1
        kept = int(c.table[0, 1])
        for x in zeroed:
            x[kept] = 0
        with_zeros = {n: torch.as_tensor(x, device="cuda").to(t[n].dtype) for n, x in zip(("k_pages", "v_pages"), zeroed)}
        got = out.clone()
        assert run(**with_zeros) == 0 and torch.equal(got, out)
    pos = torch.arange(3 * new, dtype=torch.int32, device="cuda") % new
    assert run(positions=pos) == 0
    want = out.clone()
    for r in range(3):
        falls = pos.clone()
        falls[r * new + 5] = 100
        others = [i for i in range(3 * new) if i // new != r]
        assert run(positions=falls) == 32 and torch.equal(out[others], want[others])


@pytest.mark.parametrize("Hq", [16, 17])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_padded_steps(serve, workspace, Hq, dtype):  # noqa: F811
    """Rows behind the last request are left as they were, and may hold anything."""
    import torch
    c = Pages(62, [190, 180], [70, 70], Hq=Hq, H=1, d=64, B=16, dtype=dtype)
    assert in_tiles(serve, c)
    t, err = c.tensors(), _err()
    want, want_lse = serve.attend_paged(**t, max_new=70, workspace=workspace, err=err, return_lse=True)
    for hostile in (float("nan"), float("inf")):
        q = torch.cat([t["q"], torch.full((5, Hq, 64), hostile, device="cuda", dtype=t["q"].dtype)])
        out, lse = torch.full_like(q, 6.0), torch.full((145, Hq), 6.0, device="cuda")
        serve.attend_paged(**dict(t, q=q), max_new=70, workspace=workspace, err=err, out=out, lse=lse, return_lse=True)
        assert torch.equal(out[:-5], want) and torch.equal(lse[:-5], want_lse) and bool((out[-5:] == 6).all())
        assert bool((lse[-5:] == 6).all()) and int(err) == 0


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_long_pages_offsets(serve, workspace, dtype):  # noqa: F811
    """Pages whose elements pass 2^32."""
    import torch
    S, H, B, d, n = 300_000, 8, 16, 128, 70
    k_pages, v_pages = serve.paged_cache(S, H, B, d, getattr(torch, dtype))
    slots = torch.tensor([[S - 1, 0, S - 2, 262_144, 131_073]], dtype=torch.int32, device="cuda")
    assert n * 16 > serve.attend_paged_few_rows(1, H, d, 5 * B)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    small = [p.normal_(generator=g) for p in serve.paged_cache(5, H, B, d, getattr(torch, dtype))]
    k_pages[slots[0].long()], v_pages[slots[0].long()] = small
    q = torch.randn(n, 16 * H, d, device="cuda", generator=g).to(k_pages.dtype)
    i32, err = (lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")), _err()
    a = serve.attend_paged(q, k_pages, v_pages, slots, i32([0, n]), i32([n + 5]), n, workspace, err)
    b = serve.attend_paged(q, *small, i32([[0, 1, 2, 3, 4]]), i32([0, n]), i32([n + 5]), n, workspace, err)
    assert torch.equal(a, b) and int(err) == 0


@TYPES
def test_captured(serve, workspace, d, dtype):  # noqa: F811
    """A captured prompt whose keys are shared out, replayed with other lengths beside calls of single tokens and of the
    4-bit cache over the same workspace: the results of eager calls with a workspace of their own, bit for bit."""
    import torch
    td = getattr(torch, {"f16": "float16", "bf16": "bfloat16"}[dtype])
    H, G, B, new = 2, 16, 16, 70
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    pages = [p.normal_(generator=g) for p in serve.paged_cache(400, H, B, d, td)]
    q = torch.empty(2 * new, H * G, d, device="cuda", dtype=td).normal_(generator=g)
    tables = torch.randperm(400, generator=g, device="cuda").int()[:2 * 190].view(2, 190)
    assert new * G > serve.attend_paged_few_rows(2, H, d, 190 * B)
    starts, kv, err = i32([0, new, 2 * new]), i32([2900, 700]), _err()
    codes, scales = serve.int4_cache(50, H, B, d)
    codes.fill_(0x35), scales.fill_(0.01)
    call = lambda ws: serve.attend_paged(q, *pages, tables, starts, kv, new, ws, err, return_lse=True)
    call(workspace)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(workspace)
    apart = serve.attend_workspace()
    one = q[:3].contiguous()
    for it, lens in enumerate(([2900, 700], [3040, 3000], [1, 2999], [200, 0], [1500, 1500], [3040, 70])):
        kv.copy_(i32(lens))
        starts.copy_(i32([0, new - it, 2 * new - 3 * it]))
        q.normal_(generator=g)
        singles = lambda ws: serve.attend_paged(one, *pages, tables[:, :50].contiguous(), i32([0, 1, 3]), i32([800, 500]), 2, ws, err)
        bits = lambda ws: serve.attend_int4(one, codes, scales, tables[:1, :3] % 50, i32([0, 3]), i32([40]), 3, ws, err)
        graph.replay()
        shared = [t.clone() for t in (*out, singles(workspace), bits(workspace))]
        graph.replay()
        n = 2 * new - 3 * it
        assert all(torch.equal(a[:n], b[:n]) for a, b in zip(out, shared))
        for a, b in zip(shared, (*call(apart), singles(apart), bits(apart))):
            assert torch.equal(a[:min(n, len(a))], b[:min(n, len(b))])
    assert int(err) == 0
    assert int(workspace[:4096].count_nonzero()) == 0 and int(workspace[-256:].count_nonzero()) == 0
