"""Block tables from lengths that no step could have: flagged, and nothing written outside the arrays."""
import numpy as np
import pytest

from tests.test_gpu_serve import _err, serve  # noqa: F401

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1


def _expected(cached, new, free, table, B, n_tokens):
    """As oracle.serve.block_tables, with sums cut off at 2^31 - 1 and no more than n_tokens tokens listed."""
    width, err, taken, start = table.shape[1], 0, 0, 0
    q_starts, kv = [0], []
    req, pos, rows = np.full(n_tokens, -1), np.zeros(n_tokens, int), np.full(n_tokens, -1)
    for r, (c, n) in enumerate(zip(cached, new)):
        ok = c >= 0 and n >= 0 and c + n <= width * B
        err |= 0 if ok else 8
        n = max(n, 0)
        kv.append(c + n if ok else 0)
        if ok:
            for j in range(-(-c // B), -(-(c + n) // B)):
                table[r, j] = free[taken] if taken < len(free) else -1
                err |= 0 if taken < len(free) else 16
                taken += 1
        for i in range(min(n, max(0, n_tokens - start))):
            p = c + i if ok else 0
            slot = table[r, p // B] if ok else -1
            req[start + i], pos[start + i] = r, p
            rows[start + i] = slot * B + p % B if slot >= 0 else -1
        start += n
        q_starts.append(min(start, MOST))
    return {"q_starts": q_starts, "kv_lens": kv, "token_req": req, "token_pos": pos, "token_rows": rows,
            "n_taken": [min(taken, len(free))], "err": err | (8 if start > n_tokens else 0)}


GOOD, BAD = (3, 2), (0, MOST)


@pytest.mark.parametrize("requests", [
    [GOOD, BAD], [BAD, GOOD], [GOOD, BAD, BAD, BAD, GOOD], [(MOST, MOST)] * 3 + [GOOD], [(MOST, 1), GOOD],
    [(-MOST - 1, MOST), (MOST, -MOST - 1), GOOD, (0, MOST - 6), GOOD], [BAD] * 40 + [GOOD] * 60, [GOOD] * 4095 + [BAD] * 3 + [GOOD] * 900,
    [GOOD] * 50 + [BAD] * 5000 + [GOOD], [(0, 64)] * 30 + [BAD] * 2], ids=lambda r: f"{len(r)}")
@pytest.mark.parametrize("n_tokens", [0, 7, 4001])
def test_sums_past_32_bits(serve, requests, n_tokens):  # noqa: F811
    import torch
    B, width, edge = 16, 4, 64
    cached, new = (list(x) for x in zip(*requests))
    r = np.random.default_rng(len(requests))
    table = r.permutation(len(requests) * width).reshape(-1, width).astype(np.int32)
    free = (100_000 + r.permutation(37)).astype(np.int32)
    i32 = lambda a: torch.as_tensor(np.asarray(a, np.int32), device="cuda")
    dev, err = i32(table), _err()
    names = ("q_starts", "kv_lens", "token_req", "token_pos", "token_rows", "n_taken")
    sizes = (len(requests) + 1, len(requests), n_tokens, n_tokens, n_tokens, 1)
    wide = [torch.full((n + 2 * edge,), -77, dtype=torch.int64 if name == "token_rows" else torch.int32, device="cuda")
            for name, n in zip(names, sizes)]
    out = serve.StepTables([w[edge:edge + n] for w, n in zip(wide, sizes)])
    serve.build_block_tables(i32(cached), i32(new), i32(free), dev, B, n_tokens, err, out=out)
    want = _expected(cached, new, free.tolist(), table, B, n_tokens)
    for name, w, n in zip(names, wide, sizes):
        got = w.cpu().numpy()
        assert np.array_equal(got[edge:edge + n], want[name]), name
        assert (got[:edge] == -77).all() and (got[edge + n:] == -77).all(), name
    assert np.array_equal(dev.cpu().numpy(), table) and int(err) == want["err"]
