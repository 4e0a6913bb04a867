"""Serving from the 4-bit cache, end to end on a small random model.

    python examples/serve_int4.py [--requests 5] [--steps 24]

Each request brings an image and some text.  The image's patches go through
one encoder layer whose queries and keys turn on two axes (`rope_axes`), then
image and text go through a two-layer decoder that keeps its keys and values
in 4 bits: the prompt in chunks, then one token a step, all requests in one
call per layer (`build_block_tables` once a step, `append_int4` and
`attend_int4` in each layer).  Single-token steps replay one CUDA graph.  After
each chunk and at the end, every request's cache is read back
(`hc_fetch_rotate_scatter`) and the step's attention recomputed from that in
float64.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from kv_cache_quantization_hc_gb300 import hc, serve  # noqa: E402

HIDDEN, HQ, H, D, B, GROUP, LAYERS, VOCAB = 256, 8, 2, 64, 16, 32, 2, 1000
GRID = (6, 9)                              # patches of an image
TEXT_AXES = (0,) * 16 + (1,) * 8 + (2,) * 8      # time, height and width sections of the 32 pairs
CHUNK = 128                                # prompt tokens of a request in one step: 512 query rows per cache head, attended in tiles


class Model:
    def __init__(self, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        w = lambda n, m: (torch.randn(n, m, device="cuda", generator=g) / n ** 0.5).bfloat16()
        self.embed, self.patch_qkv = w(HIDDEN, VOCAB).t().contiguous(), w(HIDDEN, 3 * HQ * D)
        self.patch_out = w(HQ * D, HIDDEN)
        self.qkv = [w(HIDDEN, (HQ + 2 * H) * D) for _ in range(LAYERS)]
        self.out = [w(HQ * D, HIDDEN) for _ in range(LAYERS)]


def encode_image(model, patches, table, err):
    """One encoder layer: queries and keys, side by side in one buffer, rotated in place by row and column."""
    n = patches.shape[0]
    at = torch.arange(n, device="cuda", dtype=torch.int32)
    where = torch.stack([at // GRID[1], at % GRID[1]])
    qkv = (patches @ model.patch_qkv).view(n, 3 * HQ, D)
    serve.rope_axes(qkv[:, :2 * HQ], where, table, (0, 1) * (D // 4), err, pairing="interleaved", out=qkv[:, :2 * HQ])
    q, k, v = (t.transpose(0, 1).float() for t in qkv.view(n, 3, HQ, D).unbind(1))
    o = torch.softmax(q @ k.transpose(1, 2) * D ** -0.5, -1) @ v
    return patches + o.transpose(0, 1).reshape(n, HQ * D).bfloat16() @ model.patch_out


def three_axes(token_pos):
    """Positions of a sequence that starts with an image: its patches by row and column at time 0, then text."""
    n, image = token_pos.shape[0], GRID[0] * GRID[1]
    text = token_pos - image + max(GRID)
    patch = torch.stack([torch.zeros_like(token_pos), token_pos // GRID[1], token_pos % GRID[1]])
    return torch.where(token_pos < image, patch, text.expand(3, n)).int().contiguous()


class Server:
    """A decoder's state: caches, block tables, free slots, lengths."""

    def __init__(self, model, n_req, max_len):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.model, self.width = model, -(-max_len // B)
        self.caches = [serve.int4_cache(n_req * self.width + 1, H, B, D, GROUP) for _ in range(LAYERS)]
        self.tables = torch.full((n_req, self.width), -1, **i32)
        self.free = torch.arange(n_req * self.width, **i32).flip(0).contiguous()
        self.cached = torch.zeros(n_req, **i32)
        self.err = torch.zeros(1, **i32)
        self.rope = serve.rotation_table(max_len, D // 2, 1e4)
        self.workspace = serve.attend_workspace()
        self.last = None                      # the last layer's rotated queries and attention

    def step(self, x, new_lens, max_new):
        """x [tokens, HIDDEN]: new_lens of them per request, in order.  Nothing here waits for the GPU."""
        s = serve.build_block_tables(self.cached, new_lens, self.free, self.tables, B, x.shape[0], self.err)
        positions = three_axes(s.token_pos)
        for w, wo, (codes, scales) in zip(self.model.qkv, self.model.out, self.caches):
            qkv = (x @ w).view(-1, HQ + 2 * H, D)
            q = serve.append_int4(qkv[:, :HQ], qkv[:, HQ:HQ + H], qkv[:, HQ + H:], s.token_rows, codes, scales,
                                  positions, self.rope, TEXT_AXES, self.err)
            o = serve.attend_int4(q, codes, scales, self.tables, s.q_starts, s.kv_lens, max_new, self.workspace, self.err)
            x = x + o.reshape(-1, HQ * D) @ wo
        self.last = q, o
        self.cached.add_(new_lens)
        # the taken slots leave the front of the free list
        self.free.copy_(self.free[(torch.arange(self.free.numel(), device="cuda") + s.n_taken) % self.free.numel()])
        ends = (s.q_starts[1:] - 1).clamp(min=0).long()
        return (x[ends] @ self.model.embed.t()).argmax(-1)


def read_back(server, request, length, layer=-1):
    """A request's keys and values out of a layer's cache, float64 [length, H, D] each."""
    codes, scales = server.caches[layer]
    blocks = -(-length // B)
    slots = server.tables[request, :blocks].long()
    k, v = (torch.zeros(blocks, B, H, D, device="cuda") for _ in range(2))
    zero = torch.zeros(blocks, dtype=torch.int32, device="cuda")
    still = torch.zeros(1, D // 2, 2, device="cuda")
    still[..., 0] = 1                         # no further rotation
    hc.hc_fetch_rotate_scatter(hc.HC_WIRE_INT4, codes[slots], scales[slots], GROUP, hc.HC_F16, still, zero, 1,
                               hc.HC_PAIR_HALF_SPLIT, torch.arange(blocks, dtype=torch.int32, device="cuda"), None, blocks,
                               k, v, hc.paged_desc(k), server.err)
    return k.view(-1, H, D)[:length].double(), v.view(-1, H, D)[:length].double()


def deviation(server, lens, new):
    """How far the last step's attention is from its cache read back, in the values' size: request r has `lens[r]`
    tokens in the cache, `new[r]` of them from that step."""
    q, o = server.last
    worst, at = 0.0, 0
    for r, (n, m) in enumerate(zip(lens, new)):
        k, v = read_back(server, r, n)
        hidden = torch.arange(n, device="cuda") > torch.arange(n - m, n, device="cuda")[:, None]
        for h in range(HQ if m else 0):
            kh, vh = k[:, h // (HQ // H)], v[:, h // (HQ // H)]
            x = (q[at:at + m, h, None].double() * kh).sum(-1) * D ** -0.5          # [m, n]
            p = torch.softmax(x.masked_fill(hidden, float("-inf")), -1)[..., None]
            want, size = (p * vh).sum(1), (p * vh.abs()).sum(1)
            worst = max(worst, float(((o[at:at + m, h].double() - want).abs() / size.clamp(min=1e-30)).max()))
        at += m
    return worst


def main(n_req=5, steps=24, seed=0, say=print):
    torch.cuda.set_device(0)
    model = Model(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    image = GRID[0] * GRID[1]
    text = [3 + 37 * i for i in range(n_req)]
    lens = [image + t for t in text]
    server = Server(model, n_req, max(lens) + steps + 1)
    axis = serve.rotation_table(max(GRID), D // 2, 100.0)
    prompts = []
    for t in text:
        patches = torch.randn(image, HIDDEN, device="cuda", generator=g).bfloat16()
        words = torch.randint(0, VOCAB, (t,), device="cuda", generator=g)
        prompts.append(torch.cat([encode_image(model, patches, axis, server.err), model.embed[words]]))

    # prompts, a chunk of each at a time; a request whose prompt has ended brings nothing more
    token = torch.zeros(n_req, dtype=torch.long, device="cuda")
    worst = 0.0
    for at in range(0, max(lens), CHUNK):
        parts = [p[at:at + CHUNK] for p in prompts]
        new = torch.tensor([len(p) for p in parts], dtype=torch.int32, device="cuda")
        token = torch.where(new > 0, server.step(torch.cat(parts), new, CHUNK), token)
        worst = max(worst, deviation(server, [min(n, at + CHUNK) for n in lens], [len(p) for p in parts]))

    # one token per request and step: a graph over the same buffers
    one = torch.ones(n_req, dtype=torch.int32, device="cuda")
    tokens = [token]
    feed = token.clone()

    def decode():
        feed.copy_(server.step(model.embed[feed], one, 1))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        decode()                              # allocations and one-time queries, before the capture
    torch.cuda.current_stream().wait_stream(side)
    tokens.append(feed.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        decode()
    for _ in range(steps - 1):
        graph.replay()
        tokens.append(feed.clone())
    assert int(server.err) == 0, f"device errors {int(server.err):#x}"

    worst = max(worst, deviation(server, [n + steps for n in lens], [1] * n_req))
    say(f"{n_req} requests of {min(lens)} to {max(lens)} prompt tokens, {steps} more each; "
        f"{server.caches[0][0].numel() * 2 * LAYERS} codes; attention against its cache: {worst:.2e} of the values' size")
    for r, row in enumerate(torch.stack(tokens, 1).tolist()):
        say(f"  request {r}: {' '.join(map(str, row[:12]))} ...")
    return worst, torch.stack(tokens, 1)


if __name__ == "__main__":
    a = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    a.add_argument("--requests", type=int, default=5)
    a.add_argument("--steps", type=int, default=24)
    a = a.parse_args()
    main(a.requests, a.steps)
