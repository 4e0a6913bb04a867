"""What tests/test_gpu_serve.py asks of attention, asked of requests with many query rows, which another kernel takes:
ranges, zeros, strides, bad lengths and slots, offsets past 32 bits."""
import numpy as np
import pytest

from oracle import serve as oserve
from tests.serve_cases import Cache
from tests.test_gpu_serve import _check_attend, _err, serve, workspace  # noqa: F401

pytestmark = pytest.mark.gpu


def _many(serve, c):  # noqa: F811
    """The cache, if all its requests have more rows than the few-rows kernel takes."""
    few = serve.attend_few_rows(len(c.kv), c.H, c.d)
    assert all(n * (c.Hq // c.H) > few for n in c.new), (few, c.new)
    return c


@pytest.mark.parametrize("scale,spread", [("f32", 1e6), ("f32", 1e-12), ("f16", 1e-4), ("f16", 3e4), ("f32", 1.0)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d,group", [(64, 32), (128, 128)])
def test_ranges(serve, workspace, scale, spread, dtype, d, group):  # noqa: F811
    """Scales and queries far from 1; scores within the 22 bits that fp16 probabilities keep whole."""
    if dtype == "f16" and spread > 1e4:
        spread = 300.0                                            # the output has to hold the values
    if dtype == "f16" and spread < 1e-6:
        spread = 1e-3
    q_scale = 30.0 if dtype == "f16" else 1e5
    c = _many(serve, Cache(61, [610, 477], [200, 130], Hq=4, H=1, d=d, B=16, group=group, scale=scale, dtype=dtype,
                           spread=spread, outliers=False, q_scale=q_scale))
    for x in (0.1, 0.001):
        _check_attend(serve, workspace, c, softmax_scale=x / (spread * q_scale))


def test_values_of_mixed_magnitude(serve, workspace):  # noqa: F811
    """Value scales that grow and shrink by orders of magnitude from one run of 32 keys to the next."""
    c = _many(serve, Cache(62, [900], [300], Hq=8, H=2, d=128, B=16, group=32, scale="f32", outliers=False))
    for j in range(900):
        c.scales[c.table[0, j // 16], 1, :, j % 16] *= 10.0 ** (j // 32 % 5 - 2)
    c.scales = oserve.round_like(c.scales, "f32")
    _check_attend(serve, workspace, c)


def test_values_of_zeros(serve, workspace):  # noqa: F811
    c = _many(serve, Cache(63, [500, 450], [400, 450], Hq=2, H=2, d=64, B=16, group=64, hostile=False))
    c.scales[:, 1] = 0
    c.q[::4] = 0
    got, _ = _check_attend(serve, workspace, c)
    assert not bool(got.any())


@pytest.mark.parametrize("d,group,scale", [(64, 32, "f16"), (128, 64, "f32")])
def test_strided_rows(serve, workspace, d, group, scale):  # noqa: F811
    """Queries out of a packed buffer, outputs into one; other rows untouched."""
    import torch
    c = _many(serve, Cache(64, [500, 190], [150, 121], Hq=8, H=2, d=d, B=32, group=group, scale=scale))
    t, err = c.tensors(), _err()
    n = t["q"].shape[0]
    packed = torch.randn(n, 12, d, device="cuda").to(torch.bfloat16)
    packed[:, 2:10] = t["q"]
    wide = torch.full((n + 2, 11, d), 7.0, dtype=torch.bfloat16, device="cuda")
    a = serve.attend_int4(t["q"], t["codes"], t["scales"], t["table"], t["q_starts"], t["kv"], 150, workspace, err)
    serve.attend_int4(packed[:, 2:10], t["codes"], t["scales"], t["table"], t["q_starts"], t["kv"], 150, workspace,
                      err, out=wide[:n, 1:9])
    assert torch.equal(wide[:n, 1:9], a) and int(err) == 0
    assert bool((wide[:, 0] == 7).all()) and bool((wide[:, 9:] == 7).all()) and bool((wide[n:] == 7).all())
    _check_attend(serve, workspace, c)


@pytest.mark.parametrize("scale", ["f16", "f32"])
def test_bad_lengths_and_slots(serve, workspace, scale):  # noqa: F811
    import torch
    new = 120
    c = _many(serve, Cache(65, [264, 250, 264], [new] * 3, Hq=4, H=1, d=64, B=16, group=32, scale=scale))
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
    zeros = t["scales"].clone()                                    # a block without a slot counts as zeros
    zeros[t["table"][0, 1].long()] = 0
    want = serve.attend_int4(t["q"], t["codes"], zeros, t["table"], t["q_starts"], t["kv"], new, workspace, _err())
    for slot in (-1, c.codes.shape[0], 2 ** 31 - 1):
        table = t["table"].clone()
        table[0, 1] = slot
        err = _err()
        run(err, table=table)
        assert int(err) == 1 and torch.equal(out[new:], good[new:]) and torch.equal(out[:new], want[:new])


def test_long_cache_offsets(serve, workspace):  # noqa: F811
    """A cache whose codes pass 4 GiB and whose rows' offsets pass 32 bits."""
    import torch
    S, H, B, d, n = 300_000, 8, 16, 128, 400
    codes, scales = serve.int4_cache(S, H, B, d)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    used = torch.randperm(S, device="cuda", generator=g)[: n // B]
    used[:4] = torch.tensor([S - 1, 0, S - 2, 262_144], device="cuda")
    assert used.unique().numel() == n // B and n > serve.attend_few_rows(1, H, d)
    q, k, v = (torch.randn(n, H, d, device="cuda", generator=g).to(torch.bfloat16) for _ in range(3))
    pos = torch.arange(n, device="cuda")
    err = _err()
    serve.append_int4(None, k, v, used[pos // B] * B + pos % B, codes, scales, None, None, None, err)
    small_c, small_s = serve.int4_cache(n // B, H, B, d)
    serve.append_int4(None, k, v, pos, small_c, small_s, None, None, None, err)
    assert torch.equal(codes[used], small_c) and torch.equal(scales[used], small_s)
    i32 = lambda a: torch.as_tensor(a, dtype=torch.int32, device="cuda")
    starts, kv = i32([0, n]), i32([n])
    a = serve.attend_int4(q, codes, scales, used.int()[None], starts, kv, n, workspace, err)
    b = serve.attend_int4(q, small_c, small_s, i32(np.arange(n // B))[None], starts, kv, n, workspace, err)
    assert torch.equal(a, b) and int(err) == 0


def test_the_limit_is_where_the_kernels_change(serve, workspace):  # noqa: F811
    """Either side of attend_few_rows, the same request within both kernels' bars."""
    for n_req in (1, 30):
        few = serve.attend_few_rows(n_req, 2, 64)
        for rows in (few, few + 1):
            kv, new = [rows + 70] + [5] * (n_req - 1), [rows] + [1] * (n_req - 1)
            _check_attend(serve, workspace, Cache(66, kv, new, Hq=2, H=2, d=64, B=16, group=32))
