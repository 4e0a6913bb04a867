"""The serving operators over a 4-bit paged cache, as workloads.

Four operators, each in a plain form (elementary torch operations in 32 bits)
and as the calls of ``kv_cache_quantization_hc_gb300.serve``:

* ``tables``: one step's block tables, token positions and cache rows from the
  requests' lengths;
* ``rope``: rotary positions with several axes (time, height, width), or its
  gradient (the rotation by the opposite angle);
* ``append``: the new tokens' queries and keys rotated, keys and values
  quantized to grouped INT4 and written to their cache rows; the cache's
  values are then read back through the fetch, as a block is when it leaves
  the 4-bit cache;
* ``attend``: attention of the new tokens over the 4-bit cache, from one token
  per request to whole prompts.

Lengths follow the quantiles of a log-uniform distribution between a case's
bounds (in an order drawn from the seed), so that a case's work is the same
for every seed.  Keys and values are N(0, 1) with 2% of the channels ten times
as large, the distribution of the ``ragged`` workload.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_ES = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step's addressing: 64 requests of the ragged workload's lengths
        {"name": "tables_decode", "op": "tables", "n_req": 64, "B": 16, "cached_lo": 200,
         "cached_hi": 25000, "new_lo": 1, "new_hi": 1},
        # an offline batch's prompts taken in at once: 4096 requests, about a million new tokens
        {"name": "tables_prompts", "op": "tables", "n_req": 4096, "B": 16, "cached_lo": 1,
         "cached_hi": 4000, "new_lo": 10, "new_hi": 1200},
        # one image's worth of queries and keys, sections per axis, out of a packed q/k/v buffer
        {"name": "rope_image", "op": "rope", "n": 1369, "H": 40, "spare": 8, "d": 128, "rot": 128,
         "axes": 3, "cyclic": False, "pairing": "half_split", "dtype": "bf16", "inverse": False},
        # the gradient of a long video's queries in 32 bits, axes interleaved, a partial rotation
        {"name": "rope_video_grad", "op": "rope", "n": 20011, "H": 32, "spare": 0, "d": 128,
         "rot": 96, "axes": 3, "cyclic": True, "pairing": "interleaved", "dtype": "f32",
         "inverse": True},
        # one decoding step of 64 requests: 64 tokens to 64 blocks
        {"name": "append_decode", "op": "append", "n_req": 64, "new": 1, "Hq": 32, "H": 8, "d": 128,
         "B": 16, "group": 32, "scale": "f16", "axes": 1, "pairing": "half_split", "dtype": "bf16"},
        # a chunk of prompts: 7 requests of 1171 tokens
        {"name": "append_chunk", "op": "append", "n_req": 7, "new": 1171, "Hq": 32, "H": 8, "d": 128,
         "B": 64, "group": 128, "scale": "f16", "axes": 3, "pairing": "half_split", "dtype": "f16"},
        # a single user's next token early in a chat: latency
        {"name": "attend_one", "op": "attend", "n_req": 1, "cached_lo": 999, "cached_hi": 999,
         "new_lo": 1, "new_hi": 1, "Hq": 32, "H": 8, "d": 128, "B": 16, "group": 32, "scale": "f16",
         "dtype": "bf16", "window": 0, "lse": True},
        # a decoding step of the ragged workload's 64 requests
        {"name": "attend_ragged", "op": "attend", "n_req": 64, "cached_lo": 200, "cached_hi": 25000,
         "new_lo": 1, "new_hi": 1, "Hq": 32, "H": 8, "d": 128, "B": 16, "group": 32, "scale": "f16",
         "dtype": "bf16", "window": 0, "lse": True},
        # long contexts with 8 query heads per cache head: the largest cache read
        {"name": "attend_long", "op": "attend", "n_req": 8, "cached_lo": 131000, "cached_hi": 131071,
         "new_lo": 1, "new_hi": 1, "Hq": 64, "H": 8, "d": 128, "B": 64, "group": 128, "scale": "f16",
         "dtype": "f16", "window": 0, "lse": True},
        # drafted tokens checked, a few per request, with a sliding window
        {"name": "attend_drafts", "op": "attend", "n_req": 37, "cached_lo": 50, "cached_hi": 9000,
         "new_lo": 2, "new_hi": 7, "Hq": 14, "H": 2, "d": 64, "B": 32, "group": 64, "scale": "f32",
         "dtype": "f16", "window": 4096, "lse": True},
        # prompts' chunks over what is cached of them, odd lengths
        {"name": "attend_chunks", "op": "attend", "n_req": 7, "cached_lo": 16, "cached_hi": 4000,
         "new_lo": 101, "new_hi": 3001, "Hq": 32, "H": 8, "d": 128, "B": 16, "group": 32,
         "scale": "f16", "dtype": "bf16", "window": 0, "lse": False},
        # one whole prompt: the largest product
        {"name": "attend_prompt", "op": "attend", "n_req": 1, "cached_lo": 0, "cached_hi": 0,
         "new_lo": 8192, "new_hi": 8192, "Hq": 32, "H": 8, "d": 128, "B": 16, "group": 32,
         "scale": "f16", "dtype": "bf16", "window": 0, "lse": False},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_attend(rng):
    d = rng.choice((64, 128))
    H = rng.choice((1, 2, 4, 8))
    c = {"op": "attend", "d": d, "H": H, "Hq": H * rng.choice((1, 2, 3, 4, 5, 7, 8)),
         "B": rng.choice((16, 32, 64, 128)), "group": rng.choice([g for g in (32, 64, 128) if g <= d]),
         "scale": rng.choice(("f16", "f16", "f32"))}
    kind = rng.choice(("decode", "drafts", "prompt"))
    c["window"] = rng.choice((0, 0, _log_int(rng, 100, 8000)))
    if kind == "prompt":
        c.update(n_req=_log_int(rng, 1, 12), new_lo=_log_int(rng, 20, 400),
                 new_hi=_log_int(rng, 400, 8192), dtype="bf16", lse=False)
        c["cached_lo"], c["cached_hi"] = rng.choice(((0, 0), (_log_int(rng, 1, 300), _log_int(rng, 300, 8000))))
    else:
        c.update(n_req=_log_int(rng, 1, 256), new_lo=1, new_hi=1 if kind == "decode" else rng.randint(2, 9),
                 cached_lo=_log_int(rng, 1, 500), cached_hi=_log_int(rng, 500, 130000),
                 dtype=rng.choice(("f16", "bf16")), lse=True)
    return c


def _attend_fits(c):
    """No more work than the listed cases, and a plain form (padded to the longest request) that fits."""
    cached, new = _lens(c)
    kv = max(a + b for a, b in zip(cached, new))
    w, most = work(c), [work(x) for x in listed() if x["op"] == "attend"]
    return (c["n_req"] * kv * c["H"] * c["d"] <= 1.1e9 and c["n_req"] * c["Hq"] * max(new) * kv <= 2.2e9
            and w["bytes"] <= max(m["bytes"] for m in most) and w["flops"] <= max(m["flops"] for m in most))


def draw(rng):
    op = rng.choice(("tables", "rope", "append", "attend", "attend", "attend"))
    if op == "tables":
        new_lo = rng.choice((1, 1, _log_int(rng, 2, 60)))
        return {"op": op, "n_req": _log_int(rng, 1, 4096), "B": rng.choice((16, 32, 64, 128)),
                "cached_lo": rng.choice((0, 1, 37)), "cached_hi": _log_int(rng, 40, 4000),
                "new_lo": new_lo, "new_hi": rng.choice((new_lo, _log_int(rng, 60, 1000)))}
    if op == "rope":
        d, dtype = rng.choice((64, 128)), rng.choice(("f32", "f16", "bf16"))
        H = rng.randint(1, 48)
        return {"op": op, "n": _log_int(rng, 1, max(2, int(80e6 / (H * d)))), "H": H, "spare": rng.choice((0, 2, 8)),
                "d": d, "rot": rng.choice((d, d, d // 2, 3 * d // 4)), "axes": rng.choice((1, 2, 3, 4)),
                "cyclic": rng.random() < 0.5, "pairing": rng.choice(("half_split", "interleaved")),
                "dtype": dtype, "inverse": rng.random() < 0.3}
    if op == "append":
        d, H = rng.choice((64, 128)), rng.choice((1, 2, 4, 8))
        new = rng.choice((1, rng.randint(2, 9), _log_int(rng, 10, 2000)))
        return {"op": op, "n_req": _log_int(rng, 1, max(2, 8192 // new)), "new": new,
                "Hq": H * rng.choice((1, 2, 3, 4, 7)), "H": H, "d": d, "B": rng.choice((16, 32, 64, 128)),
                "group": rng.choice([g for g in (32, 64, 128) if g <= d]),
                "scale": rng.choice(("f16", "f32")), "axes": rng.choice((1, 2, 3)),
                "pairing": rng.choice(("half_split", "interleaved")),
                "dtype": rng.choice(("f32", "f16", "bf16"))}
    while True:
        c = _draw_attend(rng)
        if _attend_fits(c):
            return c


# ------------------------------------------------------------------- inputs
def _quantiles(n, lo, hi):
    if lo < 1:
        return [round((hi + 1) ** ((i + 0.5) / n)) - 1 for i in range(n)] if hi > lo else [lo] * n
    return [round(lo * (hi / lo) ** ((i + 0.5) / n)) for i in range(n)]


def _lens(c):
    return _quantiles(c["n_req"], c["cached_lo"], c["cached_hi"]), _quantiles(c["n_req"], c["new_lo"], c["new_hi"])[::-1]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _pair_axis(c):
    """Axis of each rotated pair: in thirds (or as many parts as there are axes) one after another, or in turn."""
    half, axes = c["rot"] // 2, c["axes"]
    return tuple((i % axes) if c["cyclic"] else min(i * axes // half, axes - 1) for i in range(half))


def _rotation_table(n, half, base):
    theta = base ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * theta
    return torch.stack([a.cos(), a.sin()], -1).float()


def _positions(n, axes, start, g):
    """A quarter of text (all axes alike), then frames of 28 x 36 patches."""
    text = n // 4
    t = torch.arange(n, device="cuda")
    i = (t - text).clamp(min=0)
    grid = [text + i // 1008, text + i % 1008 // 36, text + i % 36, i % 7]
    pos = torch.stack([torch.where(t < text, t, grid[a]) for a in range(axes)])
    return (pos + start).to(torch.int32).contiguous()


def _outliers(H, d, g):
    m = torch.ones(H, 1, d, device="cuda")
    for h in range(H):
        m[h, 0, torch.randperm(d, generator=g, device="cuda")[: max(1, d // 42)]] = 10.0
    return m


def _quantize(x, group, scale):
    """Grouped symmetric INT4 of x [..., d]: whole numbers -7..7 and the stored scales."""
    x = x.unflatten(-1, (-1, group))
    s = x.abs().amax(-1) / 7
    s = s.to(_DT[scale]).float()
    q = torch.where(s[..., None] != 0, x / s[..., None], torch.zeros_like(x))
    return torch.clamp(torch.round(q), -7, 7).flatten(-2), s


def _cache(c, n_slots, g):
    """A layer's cache, every slot of it filled (a slot's unused rows hold what was there before)."""
    H, B, d = c["H"], c["B"], c["d"]
    codes = torch.empty((n_slots, 2, H, B, d // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((n_slots, 2, H, B, d // c["group"]), dtype=_DT[c["scale"]], device="cuda")
    m = _outliers(H, d, g)
    step = max(1, 100_000_000 // (2 * H * B * d))
    for a in range(0, n_slots, step):
        b = min(n_slots, a + step)
        x = (torch.randn((b - a, 2, H, B, d), generator=g, device="cuda") * m).to(torch.bfloat16).float()
        q, s = _quantize(x, c["group"], c["scale"])
        q = q.to(torch.int32) & 15
        codes[a:b] = (q[..., 0::2] | (q[..., 1::2] << 4)).to(torch.uint8)
        scales[a:b] = s.to(scales.dtype)
    return codes, scales


def _prepare_tables(c, g):
    cached, new = _lens(c)
    order = torch.randperm(c["n_req"], generator=g, device="cuda").tolist()
    cached, new = [cached[i] for i in order], [new[i] for i in order]
    B = c["B"]
    held = torch.tensor([-(-a // B) for a in cached], device="cuda")
    width = max(-(-(a + b) // B) for a, b in zip(cached, new))
    need = sum(-(-(a + b) // B) - -(-a // B) for a, b in zip(cached, new))
    n_held = int(held.sum())
    slots = torch.randperm(n_held + need + 5, generator=g, device="cuda").to(torch.int32)
    table = torch.full((c["n_req"], width), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda")[None] < held[:, None]] = slots[:n_held]
    return {"cached": _i32(cached), "new": _i32(new), "free": slots[n_held:].contiguous(), "table": table,
            "n_tokens": sum(new), "n_blocks": need}


def _prepare_rope(c, g):
    packed = torch.randn((c["n"], c["H"] + c["spare"], c["d"]), generator=g, device="cuda").to(_DT[c["dtype"]])
    start = int(torch.randint(0, 1000, (1,), generator=g, device="cuda"))
    return {"x": packed[:, : c["H"]], "pos": _positions(c["n"], c["axes"], start, g), "pair_axis": _pair_axis(c),
            "axis_of_pair": torch.tensor(_pair_axis(c), device="cuda"),
            "table": _rotation_table(c["n"] + 1100, c["rot"] // 2, 1e6)}


def _prepare_append(c, g):
    n, H, d, B = c["n_req"] * c["new"], c["H"], c["d"], c["B"]
    rc = dict(c, rot=d, cyclic=False)
    packed = torch.randn((n, c["Hq"] + 2 * H, d), generator=g, device="cuda")
    packed[:, c["Hq"]:] *= torch.cat([_outliers(H, d, g)[:, 0], _outliers(H, d, g)[:, 0]])
    packed = packed.to(_DT[c["dtype"]])
    q, k, v = packed.split([c["Hq"], H, H], dim=1)
    # each request's new tokens follow a few of its last block's, in blocks of its own
    first = torch.randint(0, B, (c["n_req"], 1), generator=g, device="cuda")
    width = -(-(B - 1 + c["new"]) // B)
    n_slots = c["n_req"] * width
    slots = torch.randperm(n_slots, generator=g, device="cuda").view(c["n_req"], width)
    at = first + torch.arange(c["new"], device="cuda")
    rows = (slots.gather(1, at // B) * B + at % B).flatten()
    codes, scales = _cache(c, n_slots, g)
    pool = torch.empty((2, n_slots, B, H, d), dtype=torch.float32, device="cuda")
    return {"q": q, "k": k, "v": v, "rows": rows, "codes": codes, "scales": scales, "pool": pool,
            "pos": _positions(n, c["axes"], 500, g), "pair_axis": _pair_axis(rc),
            "axis_of_pair": torch.tensor(_pair_axis(rc), device="cuda"),
            "table": _rotation_table(n + 1100, d // 2, 1e6),
            "zeros": torch.zeros(n_slots, dtype=torch.int32, device="cuda"),
            "order": torch.arange(n_slots, dtype=torch.int32, device="cuda"),
            "still": torch.tensor([1.0, 0.0], device="cuda").repeat(1, d // 2, 1).contiguous()}


def _prepare_attend(c, g):
    cached, new = _lens(c)
    order = torch.randperm(c["n_req"], generator=g, device="cuda").tolist()
    cached, new = [cached[i] for i in order], [new[i] for i in order]
    kv = [a + b for a, b in zip(cached, new)]
    held = torch.tensor([-(-a // c["B"]) for a in kv], device="cuda")
    n_slots = int(held.sum()) + 3
    width = int(held.max())
    codes, scales = _cache(c, n_slots, g)
    table = torch.full((c["n_req"], width), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda")[None] < held[:, None]] = torch.randperm(
        n_slots, generator=g, device="cuda")[: n_slots - 3].to(torch.int32)
    q = torch.randn((sum(new), c["Hq"], c["d"]), generator=g, device="cuda").to(_DT[c["dtype"]])
    return {"q": q, "codes": codes, "scales": scales, "table": table, "starts": _i32(_starts(new)),
            "kv": _i32(kv), "max_new": max(new), "max_kv": max(kv),
            "workspace": torch.zeros(32 << 20, dtype=torch.uint8, device="cuda")}


def prepare(case, seed):
    g = _gen(seed)
    s = {"tables": _prepare_tables, "rope": _prepare_rope, "append": _prepare_append,
         "attend": _prepare_attend}[case["op"]](case, g)
    s["case"] = dict(case)
    s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


# --------------------------------------------------------------- plain forms
def _plain_tables(s):
    c, B = s["case"], s["case"]["B"]
    cached, new, table = s["cached"].long(), s["new"].long(), s["table"]
    n_req, n, nb = c["n_req"], s["n_tokens"], s["n_blocks"]
    dev = table.device
    held = (cached + B - 1) // B
    need = (cached + new + B - 1) // B - held
    q_end, b_end = new.cumsum(0), need.cumsum(0)
    which = torch.arange(n_req, device=dev)
    rb = torch.repeat_interleave(which, need, output_size=nb)
    ib = torch.arange(nb, device=dev) - (b_end - need)[rb]
    table[rb, held[rb] + ib] = s["free"][:nb]
    req = torch.repeat_interleave(which, new, output_size=n)
    pos = cached[req] + torch.arange(n, device=dev) - (q_end - new)[req]
    rows = table[req, pos // B].long() * B + pos % B
    starts = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), q_end])
    return {"tables": table, "q_starts": starts.int(), "kv_lens": (cached + new).int(), "token_req": req.int(),
            "token_pos": pos.int(), "token_rows": rows, "n_taken": b_end[-1:].int()}


def _rotate(x, pos, axis_of_pair, table, pairing, inverse):
    """x [n, H, d] in 32 bits with its first 2 * pairs channels rotated."""
    half = len(axis_of_pair)
    cs = table[pos[axis_of_pair].long().t(), torch.arange(half, device=x.device)]     # [n, half, 2]
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
    if inverse:
        sin = -sin
    body, rest = x[..., : 2 * half], x[..., 2 * half:]
    if pairing == "half_split":
        a, b = body[..., :half], body[..., half:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, rest], -1)
    a, b = body[..., 0::2], body[..., 1::2]
    turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, rest], -1)


def _plain_rope(s):
    c = s["case"]
    y = _rotate(s["x"].float(), s["pos"], s["axis_of_pair"], s["table"], c["pairing"], c["inverse"])
    return y.to(_DT[c["dtype"]])


def _values(codes, scales):
    """What a 4-bit cache [..., d/2] with scales [..., d/group] stands for, in 32 bits."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    whole = ((n ^ 8).to(torch.float32) - 8).unflatten(-1, (scales.shape[-1], -1))
    return (whole * scales.float()[..., None]).flatten(-2)


def _plain_append(s):
    c = s["case"]
    q = _rotate(s["q"].float(), s["pos"], s["axis_of_pair"], s["table"], c["pairing"], False)
    k = _rotate(s["k"].float(), s["pos"], s["axis_of_pair"], s["table"], c["pairing"], False)
    whole, sc = _quantize(torch.stack([k, s["v"].float()], 1), c["group"], c["scale"])
    new = (whole.unflatten(-1, (-1, c["group"])) * sc[..., None]).flatten(-2)      # [n, 2, H, d]
    vals = _values(s["codes"], s["scales"])                                          # [slots, 2, H, B, d]
    vals[s["rows"] // c["B"], :, :, s["rows"] % c["B"]] = new
    k, v = vals[:, 0].transpose(1, 2), vals[:, 1].transpose(1, 2)
    return {"q": q.to(_DT[c["dtype"]]), "k": k.contiguous(), "v": v.contiguous()}


def _plain_attend(s):
    c, B, H = s["case"], s["case"]["B"], s["case"]["H"]
    q, kv, starts = s["q"], s["kv"].long(), s["starts"].long()
    n, G, dev = c["n_req"], c["Hq"] // c["H"], s["q"].device
    # keys and values of every request, padded to the longest
    j = torch.arange(s["max_kv"], device=dev)
    slot = s["table"].long().clamp(min=0)[:, j // B]                                # [n, kv]
    K = _values(s["codes"][slot, 0, :, j % B], s["scales"][slot, 0, :, j % B])    # [n, kv, H, d]
    V = _values(s["codes"][slot, 1, :, j % B], s["scales"][slot, 1, :, j % B])
    # queries, padded likewise
    i = torch.arange(s["max_new"], device=dev)
    new = starts[1:] - starts[:-1]
    at = (starts[:-1, None] + i).clamp(max=q.shape[0] - 1)
    Q = q.float()[at].unflatten(2, (H, G)).permute(0, 2, 3, 1, 4).flatten(2, 3)     # [n, H, G * new, d]
    x = Q @ K.permute(0, 2, 3, 1)
    x = x.unflatten(2, (G, -1)) * (1 / math.sqrt(c["d"]))                            # [n, H, G, new, kv]
    pos = (kv - new)[:, None] + i
    seen = (j <= pos[..., None]) & (i < new[:, None])[..., None]
    if c["window"]:
        seen &= j > pos[..., None] - c["window"]
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (x - m).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.flatten(2, 3) @ V.transpose(1, 2)).unflatten(2, (G, -1)) / total.clamp(min=1e-30)
    req = torch.repeat_interleave(torch.arange(n, device=dev), new, output_size=q.shape[0])
    idx = torch.arange(q.shape[0], device=dev) - starts[req]
    y = out.permute(0, 3, 1, 2, 4).flatten(2, 3)[req, idx].to(_DT[c["dtype"]])
    if not c["lse"]:
        return y
    lse = (m + total.log())[..., 0].permute(0, 3, 1, 2).flatten(2, 3)
    return {"out": y, "lse": lse[req, idx]}


# --------------------------------------------------------- the framework's calls
def _own_tables(s):
    from kv_cache_quantization_hc_gb300 import serve
    step = serve.build_block_tables(s["cached"], s["new"], s["free"], s["table"], s["case"]["B"], s["n_tokens"],
                                    s["err"])
    return {"tables": s["table"], "q_starts": step.q_starts, "kv_lens": step.kv_lens, "token_req": step.token_req,
            "token_pos": step.token_pos, "token_rows": step.token_rows, "n_taken": step.n_taken}


def _own_rope(s):
    from kv_cache_quantization_hc_gb300 import serve
    c = s["case"]
    return serve.rope_axes(s["x"], s["pos"], s["table"], s["pair_axis"], s["err"], pairing=c["pairing"],
                           inverse=c["inverse"])


def _own_append(s):
    from kv_cache_quantization_hc_gb300 import hc, serve
    c = s["case"]
    q = serve.append_int4(s["q"], s["k"], s["v"], s["rows"], s["codes"], s["scales"], s["pos"], s["table"],
                          s["pair_axis"], s["err"], pairing=c["pairing"])
    k, v = s["pool"][0], s["pool"][1]
    hc.hc_fetch_rotate_scatter(hc.HC_WIRE_INT4, s["codes"], s["scales"], c["group"], hc.DTYPE_NAMES[c["scale"]],
                               s["still"], s["zeros"], 1, hc.HC_PAIR_HALF_SPLIT, s["order"], None,
                               s["codes"].shape[0], k, v, hc.paged_desc(k), s["err"])
    return {"q": q, "k": k, "v": v}


def _own_attend(s):
    from kv_cache_quantization_hc_gb300 import serve
    c = s["case"]
    got = serve.attend_int4(s["q"], s["codes"], s["scales"], s["table"], s["starts"], s["kv"], s["max_new"],
                            s["workspace"], s["err"], window=c["window"], return_lse=c["lse"])
    return {"out": got[0], "lse": got[1]} if c["lse"] else got


def run(state):
    op = state["case"]["op"]
    if own:
        return {"tables": _own_tables, "rope": _own_rope, "append": _own_append, "attend": _own_attend}[op](state)
    return {"tables": _plain_tables, "rope": _plain_rope, "append": _plain_append, "attend": _plain_attend}[op](state)


# ---------------------------------------------------------------------- work
def work(case):
    c, op = case, case["op"]
    if op == "tables":
        cached, new = _lens(c)
        n = sum(new)
        nb = sum(-(-(a + b) // c["B"]) - -(-a // c["B"]) for a, b in zip(cached, new))
        # lengths in, starts and lengths out; per new block its slot read and written; per token 16 bytes written
        return {"bytes": c["n_req"] * 16 + nb * 8 + n * 16, "flops": 0}
    if op == "rope":
        n = c["n"] * c["H"] * c["d"]
        pos = c["n"] * c["axes"] * 4
        # the table's rows that the positions name: at most one per token and pair, or the whole table
        rows = min(c["n"], c["n"] + 1100) * (c["rot"] // 2) * 8
        return {"bytes": 2 * n * _ES[c["dtype"]] + pos + rows, "flops": 3 * c["n"] * c["H"] * c["rot"]}
    H, d, B = c["H"], c["d"], c["B"]
    row = 2 * H * (d // 2 + d // c["group"] * _ES[c["scale"]])                       # a token's K and V in the cache
    if op == "append":
        n = c["n_req"] * c["new"]
        slots = c["n_req"] * -(-(B - 1 + c["new"]) // B)
        e = _ES[c["dtype"]]
        took = n * (2 * c["Hq"] + 2 * H) * d * e + n * (row + 8 + 4 * c["axes"] + 4 * d)
        return {"bytes": took + slots * B * (row + 2 * H * d * 4), "flops": n * (3 * c["Hq"] + 6 * H) * d}
    cached, new = _lens(c)
    rows, pairs = 0, 0
    for a, b in zip(cached, new):
        w = c["window"] or a + b
        rows += min(a + b, w + b - 1)                                                # keys that some query sees
        full = max(0, a + b - w)                                                     # queries whose window is full
        full = min(b, full)
        pairs += full * w + sum(a + i + 1 for i in range(b - full))
    n = sum(new)
    held = sum(-(-(a + b) // B) for a, b in zip(cached, new))
    return {"bytes": rows * row + n * c["Hq"] * (2 * d * _ES[c["dtype"]] + (4 if c["lse"] else 0)) + held * 4,
            "flops": 4 * pairs * c["Hq"] * d}


# --------------------------------------------------- the definitions in 64 bits
def _turned64(x, s, inverse):
    """x [n, H, d] rotated pair by pair."""
    c, x = s["case"], x.double().clone()
    pairs = s["pair_axis"]
    for i, axis in enumerate(pairs):
        lo, hi = (i, i + len(pairs)) if c["pairing"] == "half_split" else (2 * i, 2 * i + 1)
        cs = s["table"][s["pos"][axis].long(), i].double()
        z = torch.complex(x[..., lo], x[..., hi]) * torch.complex(cs[:, :1], -cs[:, 1:] if inverse else cs[:, 1:])
        x[..., lo], x[..., hi] = z.real, z.imag
    return x


def _cache64(codes, scales):
    sign = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7, -8, -7, -6, -5, -4, -3, -2, -1], dtype=torch.float64,
                        device=codes.device)
    out = torch.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=torch.float64, device=codes.device)
    out[..., 0::2], out[..., 1::2] = sign[(codes % 16).long()], sign[(codes // 16).long()]
    return out * scales.double().repeat_interleave(out.shape[-1] // scales.shape[-1], -1)


def _exact_append(s):
    c = s["case"]
    vals = _cache64(s["codes"], s["scales"]).transpose(2, 3)                         # [slots, 2, B, H, d]
    new = [_turned64(s["k"], s, False), s["v"].double()]
    for kv in range(2):
        g = new[kv].reshape(-1, c["H"], c["d"] // c["group"], c["group"])
        scale = (g.abs().max(-1, keepdim=True).values / 7).to(_DT[c["scale"]]).double()
        whole = torch.where(scale > 0, g / scale, 0.0).round().clamp(-7, 7)
        vals[s["rows"] // c["B"], kv, s["rows"] % c["B"]] = (whole * scale).reshape(-1, c["H"], c["d"])
    return {"q": _turned64(s["q"], s, False), "k": vals[:, 0], "v": vals[:, 1]}


def _exact_attend(s):
    c = s["case"]
    G = c["Hq"] // c["H"]
    starts, lens = s["starts"].tolist(), s["kv"].tolist()
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for r, n in enumerate(lens):
        a, b = starts[r], starts[r + 1]
        slots = s["table"][r, : -(-n // c["B"])].long()
        last = torch.arange(n - (b - a), n, device="cuda")[:, None]
        keys = torch.arange(n, device="cuda")[None]
        hide = keys > last
        if c["window"]:
            hide = hide | (keys <= last - c["window"])
        for h in range(c["H"]):
            k, v = (_cache64(s["codes"][slots, t, h], s["scales"][slots, t, h]).reshape(-1, c["d"])[:n] for t in (0, 1))
            for m in range(h * G, h * G + G):
                x = (s["q"][a:b, m].double() @ k.t() / math.sqrt(c["d"])).masked_fill_(hide, -math.inf)
                z = torch.logsumexp(x, 1)
                out[a:b, m] = (x - z[:, None]).exp_() @ v
                lse[a:b, m] = z
    return {"out": out, "lse": lse} if c["lse"] else out


def exact(case, seed):
    if case["op"] == "tables":
        return None
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _turned64(s["x"], s, case["inverse"])
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)
