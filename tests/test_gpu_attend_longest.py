"""Attention where a request's length is near 2^31 keys: what 32 bits do not
count is flagged, and what they do is attended."""
import pytest

from tests.test_gpu_serve import serve, workspace  # noqa: F401
from tests.test_gpu_serve_paged import _err

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1024


@pytest.fixture(scope="module")
def table():
    """2^31 keys in blocks of 16, slot 0 for all but the last blocks, which are slots 1 to 255 in turn."""
    import torch
    t = torch.zeros(1, (1 << 27) - 1, dtype=torch.int32, device="cuda")
    t[:, -255:] = torch.arange(1, 256, device="cuda")
    return t


@pytest.mark.parametrize("cache", ["pages-f16", "pages-bf16", "int4"])
@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("d", [64, 128])
def test_lengths_up_to_the_longest(serve, workspace, table, cache, new, d):  # noqa: F811
    """A window at the end, against the same keys at the start of a table."""
    import torch
    H, G, B, window = 1, 16, 16, 100
    g = torch.Generator(device="cuda")
    g.manual_seed(d + new)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    if cache == "int4":
        td, stores = torch.float16, serve.int4_cache(256, H, B, d)
        stores[0].copy_(torch.randint(0, 256, stores[0].shape, generator=g, device="cuda"))
        stores[1].copy_(torch.rand(stores[1].shape, generator=g, device="cuda"))
        call, few = serve.attend_int4, serve.attend_few_rows(1, H, d)
    else:
        td = torch.float16 if cache == "pages-f16" else torch.bfloat16
        stores = [p.normal_(generator=g) for p in serve.paged_cache(256, H, B, d, td)]
        call, few = serve.attend_paged, serve.attend_paged_few_rows(1, H, d, table.numel() * B)
    assert (new * G > few) == (new > 1)
    q = torch.empty(new, H * G, d, device="cuda", dtype=td).normal_(generator=g)
    starts = i32([0, new])

    def run(blocks, length):
        out, lse, err = torch.full_like(q, 5.0), torch.full((new, H * G), 5.0, device="cuda"), _err()
        call(q, *stores, blocks, starts, i32([length]), new, workspace, err, window=window, out=out, lse=lse, return_lse=True)
        return out, lse, int(err)

    held = table.numel() * B                       # 2^31 - 16
    for length in (MOST, MOST - 1, MOST - 77, MOST - 128):
        out, lse, err = run(table, length)
        first = (length - new - window) // B // 8 * 8          # the same keys, in tiles as before
        near, near_lse, near_err = run(table[:, first:first + 64].contiguous(), length - first * B)
        assert err == near_err == 0
        # where keys are split may differ: probabilities rounded anew (2^-8 or 2^-11 of the largest value) and the outputs
        vmax = 8.0 if cache == "int4" else float(stores[1].float().abs().max())
        step = 2.0 ** -10 if td == torch.float16 else 2.0 ** -7
        assert bool(((out.float() - near.float()).abs() <= 2 * step * vmax).all())
        assert bool(((lse - near_lse).abs() <= 2.0 ** -17 * (1 + near_lse.abs())).all())
    for length in (MOST + 1, 2 ** 31 - 128, 2 ** 31 - 64, held, held + 1, 2 ** 31 - 1):
        out, lse, err = run(table, length)
        assert err == 8 and bool((out == 5).all()) and bool((lse == 5).all())
