"""Serving from the paged buffer where the numbers are at their ends: keys past
2^24, caps and factors far from 1, more queries than keys, results in place."""
import numpy as np
import pytest

from oracle import serve as oserve
from tests.paged_cases import DT, Pages
from tests.test_gpu_serve import _rope_inputs, serve, workspace  # noqa: F401
from tests.test_gpu_serve_paged import _err, check_attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [1, 300])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_bias_by_distance_at_far_positions(serve, workspace, new, dtype):  # noqa: F811
    """A window at the end of 2^25 keys (of tables that repeat their slots): what the same keys give at the start, where
    fp32 tells neighbouring positions apart.  What differs is where keys are split: half a step each of the output."""
    import torch
    B, window, far = 64, 100, 1 << 25
    c = Pages(30, [new + 2 * B], [new], Hq=4, H=2, d=64, B=B, dtype=dtype, slopes=True, hostile=False)
    t, err = c.tensors(), _err()
    t["slopes"] *= 8                                  # a key more is up to 4 less
    blocks = -(-c.kv[0] // B)
    near, near_lse = serve.attend_paged(**dict(t, block_tables=t["block_tables"][:, :blocks].contiguous(), window=window),
                                        max_new=new, workspace=workspace, err=err, return_lse=True)
    wide = torch.zeros(1, far // B + blocks, dtype=torch.int32, device="cuda")
    wide[:, far // B:] = t["block_tables"][:, :blocks]
    got, lse = serve.attend_paged(**dict(t, block_tables=wide, kv_lens=t["kv_lens"] + far, window=window), max_new=new,
                                  workspace=workspace, err=err, return_lse=True)
    assert int(err) == 0
    # probabilities in tiles (2^-8, 2^-11) on either side, and the outputs' own rounding
    step = {"f16": 2.0 ** -10, "bf16": 2.0 ** -7}[dtype]
    vmax = float(t["v_pages"].float().abs().max())
    assert bool(((got.float() - near.float()).abs() <= 2 * step * vmax).all())
    assert bool(((lse - near_lse).abs() <= 2.0 ** -17 * (1 + near_lse.abs())).all())


@pytest.mark.parametrize("new", [1, 200])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("softcap,x", [(1e-35, 1.0), (1e-20, 1.0), (1e-3, 0.3), (1.0, 300.0), (2e5, 1.0), (3e30, 1.0), (5.0, -2.0), (5.0, 0.0),
                                       (0.02, 900.0)])
def test_caps_far_from_one(serve, workspace, dtype, new, softcap, x):  # noqa: F811
    """Scores of about x times the cap, some keys hidden in each tile."""
    c = Pages(31, [200, 277], [1, new], Hq=4, H=1, d=64, B=16, dtype=dtype, softcap=softcap, outliers=False)
    check_attend(serve, workspace, c, scale=float(np.float32(x * softcap / 64)))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("mask", [dict(prefix=[20, 300]), dict(prefix=[20, 300], window=50)], ids=str)
@pytest.mark.parametrize("softcap", [0.0, 6.0])
def test_more_queries_than_keys_with_a_bias(serve, workspace, dtype, mask, softcap):  # noqa: F811
    """Positions below 0 see the prefix only, at a distance counted from -1."""
    check_attend(serve, workspace, Pages(32, [30, 300], [45, 420], Hq=4, H=2, d=64, B=16, dtype=dtype, slopes=True,
                                         softcap=softcap, **mask))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pairing,rot", [("half_split", 64), ("half_split", 32), ("interleaved", 64)])
def test_append_in_place(serve, dtype, pairing, rot):  # noqa: F811
    """Queries rotated where they lie, beside keys and values that stay as they are."""
    import torch
    n, Hq, H, d, B = 333, 6, 2, 64, 16
    r, pos, table, pa = _rope_inputs(33, n, 3, rot // 2)
    td = getattr(torch, DT[dtype])
    x = torch.as_tensor(oserve.round_like(r.standard_normal((n, Hq + 2 * H, d)), dtype), device="cuda").to(td)
    to = lambda a: torch.as_tensor(a, device="cuda")
    results = []
    for inplace in (False, True):
        pages, err, y = serve.paged_cache(30, H, B, d, td), _err(), x.clone()
        q = y[:, :Hq]
        out = serve.append_paged(q, y[:, Hq:Hq + H], y[:, Hq + H:], torch.arange(n, device="cuda"), *pages, to(pos), to(table), pa,
                                 err, pairing=pairing, q_out=q if inplace else None)
        assert int(err) == 0 and torch.equal(y[:, Hq:], x[:, Hq:])
        results.append((out.clone(),) + pages)
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_a_call_of_one_row_and_any_strides(serve, workspace):  # noqa: F811
    """One token, one head, one slot: strides that nothing is multiplied by may be anything."""
    import torch
    c = Pages(34, [9], [1], Hq=1, H=1, d=64, B=16, extra_slots=0, hostile=False)
    t, err = c.tensors(), _err()
    want = serve.attend_paged(**t, max_new=1, workspace=workspace, err=err)
    odd = lambda x, *strides: torch.as_strided(x, x.shape, strides)
    got = serve.attend_paged(**dict(t, q=odd(t["q"], 1, 3, 1), k_pages=odd(t["k_pages"], 5, 64, 7, 1),
                                    v_pages=odd(t["v_pages"], 9, 64, 1, 1)), max_new=1, workspace=workspace, err=err)
    assert torch.equal(got, want) and int(err) == 0


@pytest.mark.parametrize("dtype,d,prefix", [("bf16", 128, False), ("f16", 64, True)])
def test_ragged_lengths_shared_out(serve, workspace, dtype, d, prefix):  # noqa: F811
    """A long request among short ones, in tiles: its keys are many parts, theirs are one; some see nothing."""
    import torch
    kv = [7000, 30, 700, 0, 2500, 3, 120, 900]
    new = [70, 30, 64, 2, 0, 3, 65, 90]
    c = Pages(35, kv, new, Hq=16, H=2, d=d, B=16, dtype=dtype, prefix=[50, 0, 9000, 0, 5, 1, 100, 300] if prefix else None)
    assert 64 * 8 > serve.attend_paged_few_rows(len(kv), c.H, c.d, c.table.shape[1] * c.B)
    a, b = check_attend(serve, workspace, c), check_attend(serve, workspace, c)
    assert all(torch.equal(x, y) for x, y in zip(a, b))        # the same bits every time
    assert int(workspace[:4096].count_nonzero()) == 0 and int(workspace[-256:].count_nonzero()) == 0


@pytest.mark.parametrize("n_req,dtype", [(170, "bf16"), (300, "f16")])
def test_many_requests_in_tiles(serve, workspace, n_req, dtype):  # noqa: F811
    """More requests than are shared out, and than are put in order of their lengths, each of more rows than go in pieces."""
    r = np.random.default_rng(n_req)
    kv = [int(v) for v in r.integers(1, 200, n_req)]
    check_attend(serve, workspace, Pages(36, kv, [17 if i % 50 else 3 for i in range(n_req)], Hq=64, H=1, d=64, B=16, dtype=dtype))
