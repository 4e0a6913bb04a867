"""Serving from the 16-bit paged buffer, as workloads.

Three operators, each in a plain form (elementary torch operations in 32 bits)
and as the calls of ``kv_cache_quantization_hc_gb300.serve``:

* ``append``: the new tokens' queries and keys rotated, keys and values written
  to their rows of the paged buffer (the one that the fetch writes and the
  encoders read);
* ``attend``: attention of the new tokens over the paged buffer, from one token
  per request to whole prompts, or of tokens at given positions (those that are
  computed again after chunks were reused); with scores capped by a tanh, a bias
  that falls with the distance, a window, or a prefix that is seen as a whole;
* ``merge``: two attention results over different keys (a history in the 4-bit
  cache, recent tokens in the paged buffer) joined by their log sums.

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
def _attend_case(name, **kw):
    c = {"name": name, "op": "attend", "spread": False, "Hq": 32, "H": 8, "d": 128, "B": 16, "dtype": "bf16", "window": 0,
         "cap": 0.0, "slopes": False, "prefix": False, "lse": True}
    c.update(kw)
    return c


def listed():
    return [
        # one decoding step of 64 requests: 64 tokens to 64 rows
        {"name": "append_decode", "op": "append", "n_req": 64, "new": 1, "Hq": 32, "H": 8, "d": 128, "rot": 128,
         "B": 16, "axes": 1, "pairing": "half_split", "dtype": "bf16"},
        # a chunk of prompts, 7 requests of 1171 tokens, three axes and a partial rotation
        {"name": "append_chunk", "op": "append", "n_req": 7, "new": 1171, "Hq": 32, "H": 8, "d": 128, "rot": 96,
         "B": 64, "axes": 3, "pairing": "interleaved", "dtype": "f16"},
        # a single user's next token early in a chat: latency
        _attend_case("attend_one", n_req=1, cached_lo=999, cached_hi=999, new_lo=1, new_hi=1),
        # a decoding step of the ragged workload's 64 requests
        _attend_case("attend_ragged", n_req=64, cached_lo=200, cached_hi=25000, new_lo=1, new_hi=1),
        # long contexts with 8 query heads per cache head: the largest cache read
        _attend_case("attend_long", n_req=8, cached_lo=131000, cached_hi=131071, new_lo=1, new_hi=1, Hq=64, B=64,
                     dtype="f16"),
        # drafted tokens checked, a few per request, scores with a bias by distance
        _attend_case("attend_drafts", n_req=37, cached_lo=50, cached_hi=9000, new_lo=2, new_hi=7, Hq=14, H=2, d=64, B=32,
                     dtype="f16", slopes=True),
        # the 15% of tokens that are computed again after chunks were reused, at their places in five prompts
        _attend_case("attend_recompute", n_req=5, cached_lo=1500, cached_hi=11000, new_lo=0, new_hi=0, spread=True,
                     lse=False),
        # prompts that start with an image, seen as a whole, over a cached instruction
        _attend_case("attend_prefix", n_req=7, cached_lo=16, cached_hi=700, new_lo=401, new_hi=4001, prefix=True,
                     lse=False),
        # prompts with capped scores and a sliding window
        _attend_case("attend_capped", n_req=3, cached_lo=0, cached_hi=0, new_lo=4099, new_hi=6007, Hq=16, H=8, B=32,
                     dtype="f16", cap=50.0, window=4096, lse=False),
        # one whole prompt: the largest product
        _attend_case("attend_prompt", n_req=1, cached_lo=0, cached_hi=0, new_lo=8192, new_hi=8192, lse=False),
        # one decoding step's results over history and recent tokens: latency
        {"name": "merge_decode", "op": "merge", "n": 64, "Hq": 32, "d": 128, "dtype": "bf16"},
        # a chunk of prompts' results, odd rows
        {"name": "merge_chunk", "op": "merge", "n": 8197, "Hq": 28, "d": 128, "dtype": "f16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_attend(rng):
    H = rng.choice((1, 2, 4, 8))
    c = _attend_case("", H=H, Hq=H * rng.choice((1, 2, 3, 4, 5, 7, 8)), d=rng.choice((64, 128)),
                     B=rng.choice((16, 32, 64, 128)), dtype=rng.choice(("f16", "bf16")))
    del c["name"]
    kind = rng.choice(("decode", "drafts", "prompt", "prompt", "recompute"))
    c["window"] = rng.choice((0, 0, 0, _log_int(rng, 100, 8000)))
    c["cap"] = rng.choice((0.0, 0.0, 0.0, 20.0, 50.0))
    c["slopes"] = rng.random() < 0.2
    if kind == "prompt":
        c.update(n_req=_log_int(rng, 1, 12), new_lo=_log_int(rng, 20, 400), new_hi=_log_int(rng, 400, 8192),
                 prefix=rng.random() < 0.25, lse=rng.random() < 0.3)
        c["cached_lo"], c["cached_hi"] = rng.choice(((0, 0), (_log_int(rng, 1, 300), _log_int(rng, 300, 8000))))
    elif kind == "recompute":
        c.update(n_req=_log_int(rng, 1, 12), new_lo=0, new_hi=0, cached_lo=_log_int(rng, 60, 1000),
                 cached_hi=_log_int(rng, 1000, 16000), spread=True, lse=rng.random() < 0.3)
    else:
        c.update(n_req=_log_int(rng, 1, 256), new_lo=1, new_hi=1 if kind == "decode" else rng.randint(2, 9),
                 cached_lo=_log_int(rng, 1, 500), cached_hi=_log_int(rng, 500, 130000))
    return c


def _attend_fits(c):
    """No more work than the listed cases, and a plain form (padded to the longest request) that fits."""
    kv, new = _lens(c)
    w, most = work(c), [work(x) for x in listed() if x["op"] == "attend"]
    return (c["n_req"] * max(kv) * c["H"] * c["d"] <= 1.1e9 and c["n_req"] * c["Hq"] * max(new) * max(kv) <= 2.2e9
            and w["bytes"] <= max(m["bytes"] for m in most) and w["flops"] <= max(m["flops"] for m in most))


def draw(rng):
    op = rng.choice(("append", "merge", "attend", "attend", "attend", "attend"))
    if op == "merge":
        Hq, d = rng.randint(1, 64), rng.choice((64, 128))
        return {"op": op, "n": _log_int(rng, 1, max(2, int(29e6 / (Hq * d)))), "Hq": Hq, "d": d,
                "dtype": rng.choice(("f32", "f16", "bf16"))}
    if op == "append":
        d, H = rng.choice((64, 128)), rng.choice((1, 2, 4, 8))
        new = rng.choice((1, rng.randint(2, 9), _log_int(rng, 10, 2000)))
        return {"op": op, "n_req": _log_int(rng, 1, max(2, 8192 // new)), "new": new, "Hq": H * rng.choice((1, 2, 3, 4)),
                "H": H, "d": d, "rot": rng.choice((d, d, d // 2, 3 * d // 4)), "B": rng.choice((16, 32, 64, 128)),
                "axes": rng.choice((1, 2, 3)), "pairing": rng.choice(("half_split", "interleaved")),
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
    """Keys and queries of each request."""
    cached = _quantiles(c["n_req"], c["cached_lo"], c["cached_hi"])
    if c["spread"]:
        return cached, [-(-3 * a // 20) for a in cached]                             # 15% of them, rounded up
    new = _quantiles(c["n_req"], c["new_lo"], c["new_hi"])[::-1]
    return [a + b for a, b in zip(cached, new)], new


def _prefixes(c, kv, new):
    """Tokens that are seen as a whole: what was cached and two fifths of what is new."""
    return [a - b + 2 * b // 5 if c["prefix"] else 0 for a, b in zip(kv, new)]


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
    """Axis of each rotated pair: in as many parts as there are axes, one after another."""
    half, axes = c["rot"] // 2, c["axes"]
    return tuple(min(i * axes // half, axes - 1) for i in range(half))


def _rotation_table(n, half, base):
    theta = base ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * theta
    return torch.stack([a.cos(), a.sin()], -1).float()


def _axis_positions(n, axes, start):
    """A quarter of text (all axes alike), then frames of 28 x 36 patches."""
    text = n // 4
    t = torch.arange(n, device="cuda")
    i = (t - text).clamp(min=0)
    grid = [text + i // 1008, text + i % 1008 // 36, text + i % 36]
    pos = torch.stack([torch.where(t < text, t, grid[a]) for a in range(axes)])
    return (pos + start).to(torch.int32).contiguous()


def _outliers(H, d, g):
    """Factors of the channels, [H, d]: one in 42 is ten times as large."""
    m = torch.ones(H, d, device="cuda")
    for h in range(H):
        m[h, torch.randperm(d, generator=g, device="cuda")[: max(1, d // 42)]] = 10.0
    return m


def _pages(c, n_slots, g):
    """One of a layer's paged buffers, every row of it filled (a slot's unused rows hold what was there before)."""
    H, B, d = c["H"], c["B"], c["d"]
    pages = torch.empty((n_slots, B, H, d), dtype=_DT[c["dtype"]], device="cuda")
    m = _outliers(H, d, g)
    step = max(1, 200_000_000 // (H * B * d))
    for a in range(0, n_slots, step):
        b = min(n_slots, a + step)
        pages[a:b] = torch.randn((b - a, B, H, d), generator=g, device="cuda") * m
    return pages


def _prepare_append(c, g):
    n, H, d, B = c["n_req"] * c["new"], c["H"], c["d"], c["B"]
    packed = torch.randn((n, c["Hq"] + 2 * H, d), generator=g, device="cuda")
    packed[:, c["Hq"]:] *= torch.cat([_outliers(H, d, g), _outliers(H, d, g)])
    q, k, v = packed.to(_DT[c["dtype"]]).split([c["Hq"], H, H], dim=1)
    # each request's new tokens follow a few of its last block's, in blocks of its own
    first = torch.randint(0, B, (c["n_req"], 1), generator=g, device="cuda")
    width = -(-(B - 1 + c["new"]) // B)
    n_slots = c["n_req"] * width
    slots = torch.randperm(n_slots, generator=g, device="cuda").view(c["n_req"], width)
    at = first + torch.arange(c["new"], device="cuda")
    rows = (slots.gather(1, at // B) * B + at % B).flatten()
    return {"q": q, "k": k, "v": v, "rows": rows, "k_pages": _pages(c, n_slots, g), "v_pages": _pages(c, n_slots, g),
            "pos": _axis_positions(n, c["axes"], 500), "pair_axis": _pair_axis(c),
            "axis_of_pair": torch.tensor(_pair_axis(c), device="cuda"),
            "table": _rotation_table(n + 1100, c["rot"] // 2, 1e6)}


def _prepare_attend(c, g):
    kv, new = _lens(c)
    order = torch.randperm(c["n_req"], generator=g, device="cuda").tolist()
    kv, new = [kv[i] for i in order], [new[i] for i in order]
    held = torch.tensor([-(-a // c["B"]) for a in kv], device="cuda")
    n_slots, width = int(held.sum()) + 3, int(held.max())
    table = torch.full((c["n_req"], width), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda")[None] < held[:, None]] = torch.randperm(
        n_slots, generator=g, device="cuda")[: n_slots - 3].to(torch.int32)
    s = {"q": torch.randn((sum(new), c["Hq"], c["d"]), generator=g, device="cuda").to(_DT[c["dtype"]]),
         "k_pages": _pages(c, n_slots, g), "v_pages": _pages(c, n_slots, g), "table": table,
         "starts": _i32(_starts(new)), "kv": _i32(kv), "max_new": max(new), "max_kv": max(kv),
         "prefix": _i32(_prefixes(c, kv, new)) if c["prefix"] else None, "at": None, "slopes": None,
         "workspace": torch.zeros(32 << 20, dtype=torch.uint8, device="cuda")}
    if c["spread"]:
        at = [((torch.arange(b, device="cuda") + torch.rand(b, generator=g, device="cuda")) * (a / b)).long().clamp(max=a - 1)
              for a, b in zip(kv, new)]
        s["at"] = torch.cat(at).to(torch.int32)
    if c["slopes"]:
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, c["Hq"] + 1, device="cuda") / c["Hq"])
    return s


def _prepare_merge(c, g):
    s = {}
    for x in ("a", "b"):
        s["out_" + x] = torch.randn((c["n"], c["Hq"], c["d"]), generator=g, device="cuda").to(_DT[c["dtype"]])
        s["lse_" + x] = 5 + 2 * torch.randn((c["n"], c["Hq"]), generator=g, device="cuda")
    # a request without a history
    none = torch.arange(c["n"], device="cuda") % 16 == 5
    s["lse_a"][none], s["out_a"][none] = -math.inf, 0
    return s


def prepare(case, seed):
    s = {"append": _prepare_append, "attend": _prepare_attend, "merge": _prepare_merge}[case["op"]](case, _gen(seed))
    s["case"] = dict(case)
    s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


# --------------------------------------------------------------- plain forms
def _rotate(x, pos, axis_of_pair, table, pairing):
    """x [n, H, d] in 32 bits with its first 2 * pairs channels rotated."""
    half = len(axis_of_pair)
    cs = table[pos[axis_of_pair].long().t(), torch.arange(half, device=x.device)]     # [n, half, 2]
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
    body, rest = x[..., : 2 * half], x[..., 2 * half:]
    if pairing == "half_split":
        a, b = body[..., :half], body[..., half:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, rest], -1)
    a, b = body[..., 0::2], body[..., 1::2]
    turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, rest], -1)


def _plain_append(s):
    c, B = s["case"], s["case"]["B"]
    q, k = (_rotate(x.float(), s["pos"], s["axis_of_pair"], s["table"], c["pairing"]).to(_DT[c["dtype"]])
            for x in (s["q"], s["k"]))
    s["k_pages"][s["rows"] // B, s["rows"] % B] = k
    s["v_pages"][s["rows"] // B, s["rows"] % B] = s["v"]
    return {"q": q, "k": s["k_pages"], "v": s["v_pages"]}


def _plain_attend(s):
    c, B, H = s["case"], s["case"]["B"], s["case"]["H"]
    q, kv, starts = s["q"], s["kv"].long(), s["starts"].long()
    n, G, dev = c["n_req"], c["Hq"] // c["H"], s["q"].device
    # keys and values of every request, padded to the longest
    j = torch.arange(s["max_kv"], device=dev)
    slot = s["table"].long().clamp(min=0)[:, j // B]                                # [n, kv]
    K, V = s["k_pages"][slot, j % B].float(), s["v_pages"][slot, j % B].float()      # [n, kv, H, d]
    # queries, padded likewise
    i = torch.arange(s["max_new"], device=dev)
    new = starts[1:] - starts[:-1]
    at = (starts[:-1, None] + i).clamp(max=q.shape[0] - 1)
    pos = (kv - new)[:, None] + i if s["at"] is None else s["at"].long()[at]         # [n, new]
    Q = q.float()[at].unflatten(2, (H, G)).permute(0, 2, 3, 1, 4).flatten(2, 3)     # [n, H, G * new, d]
    x = (Q @ K.permute(0, 2, 3, 1)).unflatten(2, (G, -1))                            # [n, H, G, new, kv]
    x *= 1 / math.sqrt(c["d"])
    if c["cap"]:
        x = (x / c["cap"]).tanh_().mul_(c["cap"])
    if s["slopes"] is not None:
        x -= s["slopes"].view(H, G, 1, 1) * (pos[..., None] - j).abs()[:, None, None]
    last = pos + 1
    if s["prefix"] is not None:
        last = torch.maximum(last, s["prefix"].long()[:, None])
    seen = (j < torch.minimum(last, kv[:, None])[..., None]) & (i < new[:, None])[..., None]
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


def _plain_merge(s):
    top = torch.maximum(s["lse_a"], s["lse_b"])
    ref = top.clamp(min=-1e30)
    wa, wb = (s["lse_a"] - ref).exp(), (s["lse_b"] - ref).exp()
    total = wa + wb
    out = (s["out_a"].float() * wa[..., None] + s["out_b"].float() * wb[..., None]) / total.clamp(min=1e-30)[..., None]
    return {"out": out.to(s["out_a"].dtype), "lse": ref + total.log()}


# --------------------------------------------------------- the framework's calls
def _own_append(s):
    from kv_cache_quantization_hc_gb300 import serve
    q = serve.append_paged(s["q"], s["k"], s["v"], s["rows"], s["k_pages"], s["v_pages"], s["pos"], s["table"],
                           s["pair_axis"], s["err"], pairing=s["case"]["pairing"])
    return {"q": q, "k": s["k_pages"], "v": s["v_pages"]}


def _own_attend(s):
    from kv_cache_quantization_hc_gb300 import serve
    c = s["case"]
    got = serve.attend_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["starts"], s["kv"], s["max_new"],
                             s["workspace"], s["err"], window=c["window"], softcap=c["cap"], slopes=s["slopes"],
                             positions=s["at"], prefix_lens=s["prefix"], return_lse=c["lse"])
    return {"out": got[0], "lse": got[1]} if c["lse"] else got


def _own_merge(s):
    from kv_cache_quantization_hc_gb300 import serve
    out, lse = serve.merge_attention(s["out_a"], s["lse_a"], s["out_b"], s["lse_b"])
    return {"out": out, "lse": lse}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "attend": _own_attend, "merge": _own_merge}[op](state)
    return {"append": _plain_append, "attend": _plain_attend, "merge": _plain_merge}[op](state)


# ---------------------------------------------------------------------- work
def work(case):
    c, op, e = case, case["op"], _ES[case["dtype"]]
    d = c["d"]
    if op == "merge":
        n = c["n"] * c["Hq"]
        return {"bytes": n * (3 * d * e + 12), "flops": 3 * n * d}
    if op == "append":
        n = c["n_req"] * c["new"]
        # rows, positions and the table's rows that they name; q, k and v read and written once
        return {"bytes": n * (8 + 4 * c["axes"] + 4 * c["rot"]) + 2 * n * (c["Hq"] + 2 * c["H"]) * d * e,
                "flops": 3 * n * (c["Hq"] + c["H"]) * c["rot"]}
    kv, new = _lens(c)
    rows, pairs = 0, 0
    for a, b, pre in zip(kv, new, _prefixes(c, kv, new)):
        at = [(2 * i + 1) * a // (2 * b) for i in range(b)] if c["spread"] else range(a - b, a)
        w = c["window"] or a
        pairs += sum(max(0, min(a, max(p + 1, pre)) - max(0, p - w + 1)) for p in at)
        end = lo = 0
        for p in at:                                                                 # keys that some query sees
            lo = max(end, p - w + 1)
            end = max(end, p + 1, min(pre, a))
            rows += end - lo
    n = sum(new)
    blocks = sum(-(-a // c["B"]) for a in kv)
    extra = 4 * n * c["spread"] + 4 * c["n_req"] * (3 + c["prefix"]) + 4 * c["Hq"] * c["slopes"]
    return {"bytes": rows * 2 * c["H"] * d * e + n * c["Hq"] * (2 * d * e + (4 if c["lse"] else 0)) + blocks * 4 + extra,
            "flops": 4 * pairs * c["Hq"] * d}


# --------------------------------------------------- the definitions in 64 bits
def _turned64(x, s):
    """x [n, H, d] rotated pair by pair."""
    c, x = s["case"], x.double().clone()
    pairs = s["pair_axis"]
    for i, axis in enumerate(pairs):
        lo, hi = (i, i + len(pairs)) if c["pairing"] == "half_split" else (2 * i, 2 * i + 1)
        cs = s["table"][s["pos"][axis].long(), i].double()
        z = torch.complex(x[..., lo], x[..., hi]) * torch.complex(cs[:, :1], cs[:, 1:])
        x[..., lo], x[..., hi] = z.real, z.imag
    return x


def _exact_append(s):
    k, v = s["k_pages"].double(), s["v_pages"].double()
    k.view((-1,) + k.shape[2:]).index_copy_(0, s["rows"], _turned64(s["k"], s))
    v.view((-1,) + v.shape[2:]).index_copy_(0, s["rows"], s["v"].double())
    return {"q": _turned64(s["q"], s), "k": k, "v": v}


def _exact_attend(s):
    c = s["case"]
    G = c["Hq"] // c["H"]
    starts, lens = s["starts"].tolist(), s["kv"].tolist()
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for r, n in enumerate(lens):
        a, b = starts[r], starts[r + 1]
        slots = s["table"][r, : -(-n // c["B"])].long()
        at = torch.arange(n - (b - a), n, device="cuda") if s["at"] is None else s["at"][a:b].long()
        away = at[:, None] - torch.arange(n, device="cuda")[None]                    # how far back a key is
        hide = away < 0
        if s["prefix"] is not None:
            hide[:, : int(s["prefix"][r])] = False
        if c["window"]:
            hide |= away >= c["window"]
        for h in range(c["H"]):
            k, v = (x[slots, :, h].double().reshape(-1, c["d"])[:n] for x in (s["k_pages"], s["v_pages"]))
            for m in range(h * G, h * G + G):
                x = s["q"][a:b, m].double() @ k.t() / math.sqrt(c["d"])
                if c["cap"]:
                    x = c["cap"] * torch.tanh(x / c["cap"])
                if s["slopes"] is not None:
                    x = x - s["slopes"][m].double() * away.abs()
                x = x.masked_fill_(hide, -math.inf)
                z = torch.logsumexp(x, 1)
                out[a:b, m] = (x - z[:, None]).exp_() @ v
                lse[a:b, m] = z
    return {"out": out, "lse": lse} if c["lse"] else out


def _exact_merge(s):
    lse = torch.logaddexp(s["lse_a"].double(), s["lse_b"].double())
    parts = [torch.exp(s["lse_" + x].double() - lse)[..., None] * s["out_" + x].double() for x in ("a", "b")]
    return {"out": parts[0] + parts[1], "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "merge": _exact_merge}[case["op"]](s)
