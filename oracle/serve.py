"""Serving from a 4-bit cache: block tables, rotary positions with several
axes, the append of new tokens, and attention.

ORACLE (test infrastructure only; see the package docstring).  Attention is in
float64 from its definition.  The rotation and the append are defined in fp32
operation by operation (include/hc.h), so they are computed here in numpy
float32, whose products and sums are each rounded once, and compare bit by bit.
"""
import numpy as np

from .numerics import round_to
from .quant import int4_dequantize, int4_pack, int4_quantize, int4_unpack  # noqa: F401 (int4_quantize: for the tests' caches)


def block_tables(cached, new, free, table, B, n_tokens):
    """One step's addressing, request by request; `table` is updated."""
    q_starts, kv, req, pos, rows, taken, err = [0], [], [], [], [], 0, 0
    width = table.shape[1]
    for r, (c, n) in enumerate(zip(map(int, cached), map(int, new))):
        ok = c >= 0 and n >= 0 and c + n <= width * B
        if not ok:
            err |= 8
        n = max(n, 0)
        kv.append(c + n if ok else 0)
        q_starts.append(q_starts[-1] + n)
        if ok:
            for j in range(-(-c // B), -(-(c + n) // B)):
                if taken < len(free):
                    table[r, j] = free[taken]
                else:
                    table[r, j] = -1
                    err |= 16
                taken += 1
        for i in range(n):
            p = c + i
            slot = int(table[r, p // B]) if ok else -1
            req.append(r)
            pos.append(p if ok else 0)
            rows.append(slot * B + p % B if slot >= 0 else -1)
    if len(req) > n_tokens:
        err |= 8
    pad = max(0, n_tokens - len(req))
    return {"q_starts": np.array(q_starts, np.int32), "kv_lens": np.array(kv, np.int32),
            "token_req": np.array(req[:n_tokens] + [-1] * pad, np.int32),
            "token_pos": np.array(pos[:n_tokens] + [0] * pad, np.int32),
            "token_rows": np.array(rows[:n_tokens] + [-1] * pad, np.int64),
            "n_taken": min(taken, len(free)), "err": err}


def rotate32(x, positions, table, pair_axis, pairing, inverse=False):
    """x float32 [n, H, d] turned in fp32, product by product."""
    x = np.array(x, np.float32)
    half = len(pair_axis)
    for i, a in enumerate(pair_axis):
        lo, hi = (i, i + half) if pairing == "half_split" else (2 * i, 2 * i + 1)
        c = table[positions[a], i, 0][:, None].astype(np.float32)
        s = table[positions[a], i, 1][:, None].astype(np.float32)
        if inverse:
            s = -s
        x1, x2 = x[:, :, lo].copy(), x[:, :, hi].copy()
        x[:, :, lo] = x1 * c - x2 * s
        x[:, :, hi] = x1 * s + x2 * c
    return x


def quantize32(x, scale_dtype):
    """Groups along the last axis of x float32: (ints int8, scales float64),
    each fp32 operation as hc_append_int4 defines it."""
    x = np.asarray(x, np.float32)
    s = np.abs(x).max(-1) * (np.float32(1) / np.float32(7))
    s = round_to(s, scale_dtype).astype(np.float32)
    q = np.divide(x, s[..., None], out=np.zeros_like(x), where=s[..., None] != 0)
    return np.clip(np.rint(q), -7, 7).astype(np.int8), s.astype(np.float64)


def append(k32, v32, rows, codes, scales, B, group, scale_dtype):
    """Rotated keys and values, float32 [n, H, d], into a copy of the cache
    (codes uint8 [S, 2, H, B, d/2], scales float64 [S, 2, H, B, d/group])."""
    codes, scales = codes.copy(), np.array(scales, np.float64)
    n, H, d = k32.shape
    for kv, x in enumerate((k32, v32)):
        ints, s = quantize32(x.reshape(n, H, d // group, group), scale_dtype)
        packed = int4_pack(ints.reshape(n, H, d))
        for t, row in enumerate(rows):
            if row >= 0:
                codes[row // B, kv, :, row % B] = packed[t]
                scales[row // B, kv, :, row % B] = s[t]
    return codes, scales


def values(codes, scales):
    """What codes [..., d/2] and scales [..., d/group] stand for, float64."""
    ints = int4_unpack(codes)
    g = scales.shape[-1]
    return int4_dequantize(ints.reshape(ints.shape[:-1] + (g, -1)), np.asarray(scales, np.float64)).reshape(ints.shape)


def attend(q, codes, scales, table, q_starts, kv_lens, B, causal=True, window=0, scale=None):
    """(out, lse, weight, reach) in float64 for q [n, Hq, d].  `weight` is
    sum_j p_j |v_j| and `reach` max_j scale * sum_c |q_c k_jc| over the visible
    keys: what rounding errors of probabilities and scores are measured by."""
    n_tok, Hq, d = q.shape
    H = codes.shape[2]
    G = Hq // H
    scale = d ** -0.5 if scale is None else scale
    out, weight = np.zeros((n_tok, Hq, d)), np.zeros((n_tok, Hq, d))
    lse, reach = np.full((n_tok, Hq), -np.inf), np.zeros((n_tok, Hq))
    for r, kv in enumerate(map(int, kv_lens)):
        a, b = int(q_starts[r]), int(q_starts[r + 1])
        for t in range(a, b):
            p = kv - (b - a) + (t - a)
            hi = min(kv, p + 1) if causal else kv
            lo = max(0, p - window + 1) if window else 0
            if lo >= hi:
                continue
            j = np.arange(lo, hi)
            slots = table[r, j // B]
            for h in range(H):
                k = values(codes[slots, 0, h, j % B], scales[slots, 0, h, j % B])
                v = values(codes[slots, 1, h, j % B], scales[slots, 1, h, j % B])
                for m in range(h * G, (h + 1) * G):
                    x = scale * (k @ q[t, m])
                    top = x.max()
                    e = np.exp(x - top)
                    out[t, m] = e @ v / e.sum()
                    weight[t, m] = e @ np.abs(v) / e.sum()
                    lse[t, m] = top + np.log(e.sum())
                    reach[t, m] = abs(scale) * (np.abs(k) @ np.abs(q[t, m])).max()
    return out, lse, weight, reach


def round_like(x, dtype):
    """x rounded to 'f32', 'f16' or 'bf16'."""
    return round_to(np.asarray(x, np.float64), dtype)
