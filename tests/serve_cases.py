"""Inputs of the serving tests: small 4-bit caches with ragged requests."""
import numpy as np

from oracle import serve as oserve

DT = {"f32": "float32", "f16": "float16", "bf16": "bfloat16"}


class Cache:
    """A layer's cache with n_req requests of kv_lens tokens (new_lens of them
    queries), every row of it filled, slots in random order; rows that no
    request holds, and table entries past a request's end, are hostile:
    NaN and infinite scales, slot ids that do not exist."""

    def __init__(self, seed, kv_lens, new_lens, *, Hq, H, d, B, group, scale="f16", dtype="bf16", spread=1.0,
                 outliers=True, window=0, causal=True, q_scale=1.0, extra_slots=3, hostile=True):
        r = np.random.default_rng(seed)
        self.kv, self.new = list(kv_lens), list(new_lens)
        self.Hq, self.H, self.d, self.B, self.group = Hq, H, d, B, group
        self.scale, self.dtype, self.window, self.causal = scale, dtype, window, causal
        held = [-(-n // B) for n in self.kv]
        S = sum(held) + extra_slots
        width = max(held + [1]) + 2
        x = r.standard_normal((S, 2, H, B, d)) * spread
        if outliers:
            x[:, :, :, :, r.choice(d, 3, replace=False)] *= 10.0
        ints, s = oserve.int4_quantize(x.reshape(S, 2, H, B, d // group, group).astype(np.float32), scale_dtype=scale)
        self.codes = oserve.int4_pack(ints.reshape(S, 2, H, B, d))
        self.scales = s
        slots = r.permutation(S)
        self.table = np.full((len(self.kv), width), S + 1000, np.int32)
        used = np.zeros((S, B), bool)
        at = 0
        for i, h in enumerate(held):
            self.table[i, :h] = slots[at: at + h]
            for j in range(self.kv[i]):
                used[self.table[i, j // B], j % B] = True
            at += h
        if hostile:
            for sl, t in zip(*np.nonzero(~used)):
                self.scales[sl, :, :, t] = r.choice([np.nan, np.inf, 6e4])
            if window:  # blocks that have slid out of every query's window are gone
                for i, (n, w) in enumerate(zip(self.kv, self.new)):
                    first = max(0, n - w - window + 1)
                    self.table[i, : first // B] = -1
        self.q_starts = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        n = int(self.q_starts[-1])
        self.q = oserve.round_like(r.standard_normal((n, Hq, d)) * q_scale, dtype)

    def expected(self, scale=None):
        return oserve.attend(self.q, self.codes, self.scales, self.table, self.q_starts, self.kv, self.B,
                             self.causal, self.window, scale)

    def tensors(self, device="cuda"):
        import torch
        to = lambda a, dt: torch.as_tensor(np.ascontiguousarray(a), device=device).to(dt)
        return {"q": to(self.q, getattr(torch, DT[self.dtype])), "codes": to(self.codes, torch.uint8),
                "scales": to(self.scales, getattr(torch, DT[self.scale])), "table": to(self.table, torch.int32),
                "q_starts": to(self.q_starts, torch.int32), "kv": to(np.asarray(self.kv), torch.int32)}


def out_bar(out, weight, reach, dtype):
    """How far an attention output may be from the definition.

    With u = 2^-11, the rounding of a number to fp16: a probability times its
    value scale is rounded once, a key and a value at most once each.  A key's
    rounding moves a score by at most u * reach, the fp32 arithmetic of a
    score (d products and the correction of the codes' offset, up to 16 times
    a code of 1) by less than another u/8 * reach, and either moves the
    weights by twice that against their sum.  Then the output's rounding."""
    u = 2.0 ** -11
    half_ulp = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
    tiny = {"f16": 2.0 ** -24, "bf16": 0.0}[dtype]
    return weight * (2.5 * u + 2.5 * u * reach[..., None]) * 1.1 + half_ulp * np.abs(out) * 1.01 + tiny


def lse_bar(lse, reach):
    """A score's error as in out_bar, and fp32's own on the sum."""
    return 1.25 * 2.0 ** -11 * reach + 2.0 ** -18 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0)))
