"""Cached chunks reused in another order, end to end on a small random model.

    python examples/reuse_chunks.py [--requests 3] [--steps 12]

A few documents go through a three-layer decoder, each by itself from position
0, and their keys and values are encoded to FP8.  Then requests come, each an
opening, the documents in an order of its own and a question.  The documents'
blocks are fetched with their keys turned to where they now stand
(`hc_fetch_rotate_scatter`).  The first layer runs over all tokens; the tokens
whose result moved furthest from the cached one (`hc_drift_select`) and those
that no document has go through the other layers as well: `append_paged` writes
their keys and values between the fetched ones and `attend_paged` attends from
their positions.  Then each request answers, one token a step, by a CUDA graph.
At last the requests' first blocks leave the pages for the 4-bit cache
(`hc_encode_int4`), and further steps attend both (`attend_int4`,
`attend_paged`) and join the results (`merge_attention`).  After each stage the
last layer's attention is recomputed from what its caches hold in float64.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from kv_cache_quantization_hc_gb300 import hc, serve  # noqa: E402

HIDDEN, HQ, H, D, B, GROUP, LAYERS, VOCAB = 256, 8, 2, 64, 16, 32, 3, 1000
DOCUMENTS = (96, 240, 64)                  # tokens of each, whole blocks
OPENING = 32
AXES = (0,) * (D // 2)
BASE = 1e4


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


class Decoder:
    """A model, its pages and what a step needs."""

    def __init__(self, n_req, max_len, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        w = lambda n, m: (torch.randn(n, m, device="cuda", generator=g) / n ** 0.5).bfloat16()
        self.embed = w(HIDDEN, VOCAB).t().contiguous()
        self.qkv = [w(HIDDEN, (HQ + 2 * H) * D) for _ in range(LAYERS)]
        self.out = [w(HQ * D, HIDDEN) for _ in range(LAYERS)]
        self.width = -(-max_len // B)
        slots = n_req * self.width + sum(DOCUMENTS) // B
        self.k, self.v = serve.paged_cache(slots, H, B, D, n_layers=LAYERS)
        self.desc = hc.paged_desc(self.k)
        self.free = torch.arange(slots, dtype=torch.int32, device="cuda").flip(0).contiguous()
        self.rope = serve.rotation_table(max_len, D // 2, BASE)
        self.workspace, self.err = serve.attend_workspace(), i32([0])
        self.history = None                # (codes, scales, tables, lengths, blocks) of what has left the pages
        self.last = None                   # the last layer's queries, their positions, its attention

    def tables_for(self, cached, new, tables, n_tokens):
        s = serve.build_block_tables(cached, new, self.free, tables, B, n_tokens, self.err)
        self.free.copy_(self.free[(torch.arange(self.free.numel(), device="cuda") + s.n_taken) % self.free.numel()])
        return s

    def layer(self, i, x, rows, at, tables, starts, kv, max_new):
        """x [tokens, HIDDEN] at positions `at` and rows `rows` through layer i."""
        qkv = (x @ self.qkv[i]).view(-1, HQ + 2 * H, D)
        q = serve.append_paged(qkv[:, :HQ], qkv[:, HQ:HQ + H], qkv[:, HQ + H:], rows, self.k[i], self.v[i], at[None], self.rope,
                               AXES, self.err)
        if self.history is None:
            o = serve.attend_paged(q, self.k[i], self.v[i], tables, starts, kv, max_new, self.workspace, self.err, positions=at)
        else:
            codes, scales, old, lens, gone = self.history
            a = serve.attend_int4(q, codes[i], scales[i], old, starts, lens, max_new, self.workspace, self.err, causal=False,
                                  return_lse=True)
            b = serve.attend_paged(q, self.k[i], self.v[i], tables[:, gone:], starts, kv - lens, max_new, self.workspace,
                                   self.err, return_lse=True)
            o, _ = serve.merge_attention(*a, *b, out=a[0])
        self.last = q, at, o
        return x + o.reshape(-1, HQ * D) @ self.out[i]

    def kv_of(self, layer, slots):
        """A layer's keys and values in these slots, float64 [tokens, H, D]."""
        return [p[layer][slots.long()].reshape(-1, H, D).double() for p in (self.k, self.v)]

    def read_history(self, r):
        """The same of what has left the last layer's pages, decoded."""
        codes, scales, old, _, gone = self.history
        at = old[r].long()
        k, v = (torch.zeros(gone, B, H, D, device="cuda") for _ in range(2))
        still = torch.zeros(1, D // 2, 2, device="cuda")
        still[..., 0] = 1
        hc.hc_fetch_rotate_scatter(hc.HC_WIRE_INT4, codes[-1][at], scales[-1][at], GROUP, hc.HC_F16, still, i32([0] * gone), 1,
                                   hc.HC_PAIR_HALF_SPLIT, i32(list(range(gone))), None, gone, k, v, hc.paged_desc(k), self.err)
        return [p.view(-1, H, D).double() for p in (k, v)]

    def deviation(self, tables, counts, lens, layer=-1):
        """How far the last attention, that of `layer`, is from its caches read back, in the values' size: request r
        has lens[r] keys and counts[r] queries."""
        q, at, o = self.last
        worst, t = 0.0, 0
        gone = 0 if self.history is None else self.history[4]
        for r, (m, n) in enumerate(zip(counts, lens)):
            k, v = self.kv_of(layer, tables[r, gone:-(-n // B)])
            if gone:
                k, v = (torch.cat(both) for both in zip(self.read_history(r), (k, v)))
            hidden = torch.arange(n, device="cuda") > at[t:t + m, None]
            for h in range(HQ):
                kh, vh = k[:n, h // (HQ // H)], v[:n, h // (HQ // H)]
                p = torch.softmax((q[t:t + m, h].double() @ kh.t() * D ** -0.5).masked_fill(hidden, float("-inf")), -1)
                worst = max(worst, float(((o[t:t + m, h].double() - p @ vh).abs() / (p @ vh.abs()).clamp(min=1e-30)).max()))
            t += m
        return worst


def encode_documents(dec, words):
    """The documents by themselves: their FP8 wire, and their hidden states behind the first layer."""
    n, blocks = sum(DOCUMENTS), sum(DOCUMENTS) // B
    tables = torch.full((len(DOCUMENTS), max(DOCUMENTS) // B), -1, dtype=torch.int32, device="cuda")
    new = i32(DOCUMENTS)
    s = dec.tables_for(torch.zeros_like(new), new, tables, n)
    x = dec.embed[words]
    for i in range(LAYERS):
        x = dec.layer(i, x, s.token_rows, s.token_pos, tables, s.q_starts, s.kv_lens, max(DOCUMENTS))
        first = x if i == 0 else first
    codes_shape, _, scales_shape = hc.wire_shapes(LAYERS, blocks, H, B, D, hc.HC_WIRE_FP8)
    codes, scales = torch.empty(codes_shape, dtype=torch.uint8, device="cuda"), torch.empty(scales_shape, device="cuda")
    slots = torch.cat([tables[c, :m // B] for c, m in enumerate(DOCUMENTS)])
    hc.hc_encode_fp8(dec.k, dec.v, dec.desc, slots, None, blocks, codes, scales, dec.err)
    return codes, scales, first


def main(n_req=3, steps=12, seed=0, say=print):
    torch.cuda.set_device(0)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    blocks, n_doc = sum(DOCUMENTS) // B, sum(DOCUMENTS)
    lens = [OPENING + n_doc + 5 + 13 * r for r in range(n_req)]
    dec = Decoder(n_req, max(lens) + 2 * steps + 1, seed)
    words = torch.randint(0, VOCAB, (n_doc,), device="cuda", generator=g)
    codes, scales, cached_hidden = encode_documents(dec, words)
    begin = [sum(DOCUMENTS[:c]) for c in range(len(DOCUMENTS))]

    # the requests' tokens, slots and fetched blocks
    tables = torch.full((n_req, dec.width), -1, dtype=torch.int32, device="cuda")
    new = i32(lens)
    s = dec.tables_for(torch.zeros_like(new), new, tables, sum(lens))
    prompts, docs = [], []
    for r, n in enumerate(lens):
        order = torch.randperm(len(DOCUMENTS), generator=torch.Generator().manual_seed(seed + r)).tolist()
        at = OPENING
        where, delta = [0] * len(DOCUMENTS), [0] * len(DOCUMENTS)
        docs.append(torch.cat([torch.arange(begin[c], begin[c] + DOCUMENTS[c], device="cuda") for c in order]))
        for c in order:
            where[c], delta[c] = at // B, at
            at += DOCUMENTS[c]
        turns = torch.empty(len(DOCUMENTS), D // 2, 2, device="cuda")
        hc.hc_build_delta_sincos(i32(delta), len(DOCUMENTS), D, BASE, None, turns)
        dst = torch.cat([tables[r, where[c]:where[c] + m // B] for c, m in enumerate(DOCUMENTS)])
        which = i32([c for c, m in enumerate(DOCUMENTS) for _ in range(m // B)])
        hc.hc_fetch_rotate_scatter(hc.HC_WIRE_FP8, codes, scales, 0, 0, turns, which, len(DOCUMENTS), hc.HC_PAIR_HALF_SPLIT, dst,
                                   None, blocks, dec.k, dec.v, dec.desc, dec.err)
        fresh = torch.randint(0, VOCAB, (n - n_doc,), device="cuda", generator=g)
        prompts.append(torch.cat([fresh[:OPENING], words[docs[-1]], fresh[OPENING:]]))

    # the first layer over all tokens, the others over those that moved
    x = dec.layer(0, dec.embed[torch.cat(prompts)], s.token_rows, s.token_pos, tables, s.q_starts, s.kv_lens, max(lens))
    worst = dec.deviation(tables, lens, lens, 0)
    starts = [sum(lens[:r]) for r in range(n_req)]
    doc_hidden = torch.stack([x[a + OPENING:a + OPENING + n_doc] for a in starts])
    _, moved = hc.drift_select(torch.stack([cached_hidden[d] for d in docs]), doc_hidden)
    chosen = []
    for r, n in enumerate(lens):
        every = torch.arange(n, device="cuda")
        chosen.append(starts[r] + torch.cat([every[:OPENING], OPENING + moved[r].long(), every[OPENING + n_doc:]]))
    counts = [len(c) for c in chosen]
    pick = torch.cat(chosen)
    x, rows, at = x[pick], s.token_rows[pick], s.token_pos[pick]
    q_starts = i32([sum(counts[:r]) for r in range(n_req + 1)])
    for i in range(1, LAYERS):
        x = dec.layer(i, x, rows, at, tables, q_starts, s.kv_lens, max(counts))
    worst = max(worst, dec.deviation(tables, counts, lens))
    token = (x[(q_starts[1:] - 1).long()] @ dec.embed.t()).argmax(-1)

    # one token per request and step: a graph over the same buffers
    cached, one = new.clone(), torch.ones_like(new)
    feed, tokens = token.clone(), [token]

    def decode():
        s = dec.tables_for(cached, one, tables, n_req)
        x = dec.embed[feed]
        for i in range(LAYERS):
            x = dec.layer(i, x, s.token_rows, s.token_pos, tables, s.q_starts, s.kv_lens, 1)
        cached.add_(one)
        feed.copy_((x @ dec.embed.t()).argmax(-1))

    def answer():
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            decode()                          # one-time queries, before the capture
        torch.cuda.current_stream().wait_stream(side)
        tokens.append(feed.clone())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            decode()
        for _ in range(steps - 1):
            graph.replay()
            tokens.append(feed.clone())
        return graph

    graph = answer()
    worst = max(worst, dec.deviation(tables, [1] * n_req, [n + steps for n in lens]))

    # the first blocks of all requests to 4 bits, and further answers over both caches
    gone = (OPENING + n_doc) // B
    left = tables[:, :gone].reshape(-1).contiguous()
    codes_shape, _, scales_shape = hc.wire_shapes(LAYERS, n_req * gone, H, B, D, hc.HC_WIRE_INT4, GROUP)
    old_codes = torch.empty(codes_shape, dtype=torch.uint8, device="cuda")
    old_scales = torch.empty(scales_shape, dtype=torch.float16, device="cuda")
    hc.hc_encode_int4(dec.k, dec.v, dec.desc, left, None, n_req * gone, GROUP, hc.HC_F16, old_codes, old_scales, dec.err)
    dec.k[:, left.long()], dec.v[:, left.long()] = float("nan"), float("nan")         # nothing reads them any more
    dec.history = (old_codes, old_scales, i32(list(range(n_req * gone))).view(n_req, gone), i32([gone * B] * n_req), gone)
    graph = answer()
    worst = max(worst, dec.deviation(tables, [1] * n_req, [n + 2 * steps for n in lens]))
    del graph
    assert int(dec.err) == 0, f"device errors {int(dec.err):#x}"

    say(f"{n_req} requests of {min(lens)} to {max(lens)} tokens, {n_doc} of them fetched and {moved.shape[1]} of those computed "
        f"again; {2 * steps} more each, the last {steps} over 4-bit blocks and pages; attention against its caches: {worst:.2e} "
        f"of the values' size")
    for r, row in enumerate(torch.stack(tokens, 1).tolist()):
        say(f"  request {r}: {' '.join(map(str, row[:12]))} ...")
    return worst, torch.stack(tokens, 1)


if __name__ == "__main__":
    a = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    a.add_argument("--requests", type=int, default=3)
    a.add_argument("--steps", type=int, default=12)
    a = a.parse_args()
    main(a.requests, a.steps)
