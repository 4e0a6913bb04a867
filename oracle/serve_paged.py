"""Serving from the paged buffer: append, attention with its masks and score
forms, and the merge of two results.

ORACLE (test infrastructure only; see the package docstring).  Attention and
merge are in float64 from their definitions (include/hc.h), key by key; the
rotation of the append is fp32 operation by operation (oracle/serve.py).
"""
import numpy as np

from .serve import rotate32, round_like


def append(k, v, rows, k_pages, v_pages, dtype, positions=None, table=None, pair_axis=None, pairing="half_split"):
    """Copies of the pages [S, B, H, d] (float64) with k, v [n, H, d] at rows >= 0, keys rotated."""
    k_pages, v_pages = np.array(k_pages, np.float64), np.array(v_pages, np.float64)
    if table is not None:
        k = round_like(rotate32(np.asarray(k, np.float32), positions, table, pair_axis, pairing), dtype)
    B = k_pages.shape[1]
    for t, row in enumerate(rows):
        if row >= 0:
            k_pages[row // B, row % B], v_pages[row // B, row % B] = k[t], v[t]
    return k_pages, v_pages


def attend(q, k_pages, v_pages, table, q_starts, kv_lens, causal=True, window=0, scale=None, softcap=0.0, slopes=None,
           positions=None, prefix_lens=None):
    """(out, lse, weight, reach, far) in float64 for q [n, Hq, d].  `weight` is
    sum_j p_j |v_j|, `reach` max_j scale * sum_c |q_c k_jc| and `far` the largest
    bias over the visible keys: what rounding errors are measured by."""
    n_tok, Hq, d = q.shape
    B, H = k_pages.shape[1:3]
    G = Hq // H
    scale = d ** -0.5 if scale is None else scale
    out, weight = np.zeros((n_tok, Hq, d)), np.zeros((n_tok, Hq, d))
    lse, reach, far = np.full((n_tok, Hq), -np.inf), np.zeros((n_tok, Hq)), np.zeros((n_tok, Hq))
    for r, kv in enumerate(map(int, kv_lens)):
        a, b = int(q_starts[r]), int(q_starts[r + 1])
        for t in range(a, b):
            p = max(kv - (b - a) + (t - a) if positions is None else int(positions[t]), -1)
            j = np.arange(kv)
            seen = np.ones(kv, bool)
            if causal:
                seen = j <= p
                if prefix_lens is not None:
                    seen |= j < prefix_lens[r]
            if window:
                seen &= j > p - window
            j = j[seen]
            if not len(j):
                continue
            slots = table[r, j // B]
            for h in range(H):
                k, v = (np.asarray(x[slots, j % B, h], np.float64) for x in (k_pages, v_pages))
                for m in range(h * G, (h + 1) * G):
                    x = scale * (k @ q[t, m])
                    if softcap:
                        x = softcap * np.tanh(x / softcap)
                    if slopes is not None:
                        x = x - float(slopes[m]) * np.abs(p - j)
                        far[t, m] = abs(float(slopes[m])) * np.abs(p - j).max()
                    top = x.max()
                    e = np.exp(x - top)
                    out[t, m] = e @ v / e.sum()
                    weight[t, m] = e @ np.abs(v) / e.sum()
                    lse[t, m] = top + np.log(e.sum())
                    reach[t, m] = abs(scale) * (np.abs(k) @ np.abs(q[t, m])).max()
    return out, lse, weight, reach, far


def merge(out_a, lse_a, out_b, lse_b):
    """(out, lse) of two results; a side with lse -inf counts for nothing."""
    top = np.maximum(lse_a, lse_b)
    ref = np.where(np.isinf(top), 0.0, top)
    w = [np.exp(np.asarray(x, np.float64) - ref) for x in (lse_a, lse_b)]
    total = w[0] + w[1]
    out = sum(np.where(x[..., None] > 0, x[..., None] * np.where(x[..., None] > 0, o, 0.0), 0.0)
              for x, o in zip(w, (out_a, out_b)))
    with np.errstate(divide="ignore"):
        return out / np.where(total > 0, total, 1.0)[..., None], np.where(total > 0, ref + np.log(total), -np.inf)
