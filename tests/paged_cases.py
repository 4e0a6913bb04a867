"""Inputs of the tests of serving from the paged buffer, and how far results may be off."""
import numpy as np

from oracle import serve as oserve
from oracle import serve_paged as opaged

DT = {"f32": "float32", "f16": "float16", "bf16": "bfloat16"}
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}       # half a step, relative


class Pages:
    """A layer's pages with requests of kv_lens tokens, new_lens of them
    queries; slots in random order.  Rows that no request holds are hostile (NaN
    and infinite), and so are table entries past a request's end (slots that do
    not exist) and, with a window, the blocks that it has left."""

    def __init__(self, seed, kv_lens, new_lens, *, Hq, H, d, B, dtype="bf16", causal=True, window=0, softcap=0.0,
                 slopes=False, positions=None, prefix=None, spread=1.0, q_scale=1.0, outliers=True, extra_slots=3,
                 hostile=True):
        r = np.random.default_rng(seed)
        self.kv, self.new = list(kv_lens), list(new_lens)
        self.Hq, self.H, self.d, self.B, self.dtype = Hq, H, d, B, dtype
        held = [-(-n // B) for n in self.kv]
        S = sum(held) + extra_slots
        x = r.standard_normal((2, S, B, H, d)) * spread
        if outliers:
            x[..., r.choice(d, 3, replace=False)] *= 10.0
        x = oserve.round_like(x, dtype)
        self.table = np.full((len(self.kv), max(held + [1]) + 2), S + 1000, np.int32)
        used = np.zeros((S, B), bool)
        slots = iter(r.permutation(S))
        for i, h in enumerate(held):
            self.table[i, :h] = [next(slots) for _ in range(h)]
            for j in range(self.kv[i]):
                used[self.table[i, j // B], j % B] = True
        if hostile:
            x[:, ~used] = r.choice([np.nan, np.inf, -np.inf, 3e4], (2, int((~used).sum()), H, d))
            if window and positions is None and prefix is None:
                for i, (n, w) in enumerate(zip(self.kv, self.new)):
                    self.table[i, : max(0, n - w - window + 1) // B] = -1
        self.k, self.v = x
        self.q_starts = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        n = int(self.q_starts[-1])
        self.q = oserve.round_like(r.standard_normal((n, Hq, d)) * q_scale, dtype)
        self.scores = dict(causal=causal, window=window, softcap=softcap,
                           slopes=np.float32(2.0) ** np.float32(-8.0 * np.arange(1, Hq + 1) / Hq) if slopes else None,
                           positions=None if positions is None else np.asarray(positions, np.int32),
                           prefix_lens=None if prefix is None else np.asarray(prefix, np.int32))

    def expected(self, scale=None):
        return opaged.attend(self.q, self.k, self.v, self.table, self.q_starts, self.kv, scale=scale, **self.scores)

    def tensors(self, device="cuda"):
        import torch
        to = lambda a, dt: torch.as_tensor(np.ascontiguousarray(a), device=device).to(dt)
        td = getattr(torch, DT[self.dtype])
        t = {"q": to(self.q, td), "k_pages": to(self.k, td), "v_pages": to(self.v, td), "block_tables": to(self.table, torch.int32),
             "q_starts": to(self.q_starts, torch.int32), "kv_lens": to(np.asarray(self.kv), torch.int32)}
        for name, dt in (("slopes", torch.float32), ("positions", torch.int32), ("prefix_lens", torch.int32)):
            t[name] = None if self.scores[name] is None else to(self.scores[name], dt)
        return dict(t, **{k: self.scores[k] for k in ("causal", "window", "softcap")})


def score_error(reach, far, d, softcap=0.0):
    """A score's error: d products, exact in fp32, summed in fp32, whose adders
    may cut off instead of rounding: 2^-23 of the sum of magnitudes each; then
    the scaling, the bias and the difference from the reference, rounded at 2^-24
    of at most the score's and the bias' size each, the cap to 2^-22 of itself."""
    return reach * d * 2.0 ** -23 + (reach + far) * 2.0 ** -21 + softcap * 2.0 ** -21


def out_bar(out, weight, reach, far, vmax, d, dtype, few, softcap=0.0):
    """How far an attention output may be from the definition: the scores'
    errors move the weights by twice that against their sum; exponentials and
    sums are good to 2^-20; probabilities are rounded to the values' type (few
    rows: to 16 bits, the upper 8 cut off and the rest rounded, or 22); in fp16
    what is below 2^-14 is off by up to 2^-25, where the largest stands at 2^3 or
    more (11.5 less 5 and at most 3.5; few rows: at 2^15), so n <= 512 keys lose at
    most 2^-28 * 512 = 2^-19 of the largest value; and the output is rounded."""
    u = {"bf16": 2.0 ** -15, "f16": 2.0 ** -21}[dtype] if few else HALF[dtype]
    lost = (2.0 ** -31 if few else 2.0 ** -19) * vmax if dtype == "f16" else 0.0
    tiny = 2.0 ** -24 if dtype == "f16" else 0.0
    return (weight * (u + 2 * score_error(reach, far, d, softcap)[..., None] + 2.0 ** -20) * 1.05 + HALF[dtype] * np.abs(out) * 1.01
            + lost + tiny)


def lse_bar(lse, reach, far, d, softcap=0.0):
    """A score's error, and fp32's own on the sum."""
    return score_error(reach, far, d, softcap) + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0)))
