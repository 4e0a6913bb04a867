"""Serving from the 4-bit cache and from the paged buffer: the calls of include/hc.h on torch tensors.

A layer's cache is an INT4 wire over its slots, codes [num_slots, 2, H, B,
d/2] and scales [num_slots, 2, H, B, d/group] (`int4_cache` makes one; the
codes and scales of hc_encode_int4 with one layer are one too).  One step of
a decoder:

  step = build_block_tables(cached_lens, new_lens, free_slots, tables, B, n_tokens, err)
  per layer:
    q = append_int4(q, k, v, step.token_rows, codes, scales, positions, table, pair_axis, err)
    o = attend_int4(q, codes, scales, tables, step.q_starts, step.kv_lens, max_new, workspace, err)

The paged buffer that the fetch writes is one to serve from too: K and V pages
[num_slots, B, H, d] in 16 bits (`paged_cache` makes them), with the same block
tables, through append_paged and attend_paged.  Results over both are joined by
merge_attention.

Every call takes its tensors on the GPU, enqueues its kernel on `stream`
(default: torch's current stream; else a torch.cuda.Stream or a cudaStream_t as
an integer) and returns without synchronising; tensors that it makes are
allocated on that stream.  An argument it cannot take raises.  What only the device sees (a slot, length or
position out of range) sets bits HC_DEVERR_* in `err`, an int32 tensor that
the caller zeroes and reads.  Tensors used on another stream than the one
they were allocated on are the caller's to record (`Tensor.record_stream`).
"""
import os

import torch

from . import build, hc

if not os.path.exists(build.BINDING):
    raise RuntimeError(f"{build.BINDING} is missing: build it with `python -c \"import __graft_entry__ as g; "
                       "g.build()\"` (the CUDA path has no fallback)")
from . import _serve  # noqa: E402

StepTables = _serve.StepTables


def int4_cache(num_slots, H, B, d, group=32, scale_dtype="f16", n_layers=None, device="cuda"):
    """Codes and scales of an empty 4-bit cache; with n_layers, one leading dimension more."""
    lead = () if n_layers is None else (n_layers,)
    sdt = {"f16": torch.float16, "f32": torch.float32}[scale_dtype]
    return (torch.zeros(lead + (num_slots, 2, H, B, d // 2), dtype=torch.uint8, device=device),
            torch.zeros(lead + (num_slots, 2, H, B, d // group), dtype=sdt, device=device))


def rotation_table(n_positions, pairs, rope_base, device="cuda", stream=None):
    """(cos, sin) of positions 0..n_positions-1 for `pairs` pairs, f32
    [n_positions, pairs, 2] (hc_build_delta_sincos)."""
    at = torch.arange(n_positions, dtype=torch.int32, device=device)
    table = torch.empty((n_positions, pairs, 2), dtype=torch.float32, device=device)
    hc.hc_build_delta_sincos(at, n_positions, 2 * pairs, rope_base, None, table, stream)
    return table


def attend_workspace(device="cuda"):
    """A workspace for attend_int4 and attend_paged (zeroed; each call leaves it
    ready for the next).  Calls that may run at the same time need one each."""
    size = max(hc.lib().hc_attend_int4_workspace(), hc.lib().hc_attend_paged_workspace())
    return torch.zeros(size, dtype=torch.uint8, device=device)


def attend_few_rows(n_req, n_kv_heads, d):
    """hc_attend_int4_few_rows: the largest number of query rows of a request (new
    tokens times query heads per cache head) that attend_int4 takes as few in a
    call of n_req requests; others are attended in fp16 tiles."""
    rows = hc.lib().hc_attend_int4_few_rows(n_req, n_kv_heads, d)
    if rows < 0:
        hc._check("hc_attend_int4_few_rows", rows)
    return rows


def build_block_tables(cached_lens, new_lens, free_slots, block_tables, block_size, n_tokens, err,
                       out=None, stream=None):
    """hc_build_block_tables: writes the new blocks' slots into block_tables
    (int32 [n_req, width], updated in place) and returns the StepTables
    (`out`: one to write into, its token arrays of n_tokens entries)."""
    return _serve.build_block_tables(cached_lens, new_lens, free_slots, block_tables, block_size, n_tokens, err,
                                     out, stream)


def rope_axes(x, positions, table, pair_axis, err, pairing="half_split", inverse=False, out=None,
              stream=None):
    """hc_rope_axes: x [n_tokens, n_heads, d] with its pairs turned.

    positions int32 [n_axes, n_tokens]; table [n_positions, pairs, 2]; pair_axis:
    the axis of each pair.  inverse=True turns back, which is also the gradient
    of the rotation.  out=x rotates in place; queries and keys that lie in one
    packed buffer are one call on the view of both."""
    return _serve.rope_axes(x, positions, table, pair_axis, err, pairing, inverse, out, stream)


def append_int4(q, k, v, token_rows, codes, scales, positions, table, pair_axis, err,
                pairing="half_split", q_out=None, stream=None, wire_scales=False):
    """hc_append_int4: k, v [n_tokens, H, d] into the cache at token_rows
    (int64), keys rotated; returns the rotated q (None for q None).  table
    None: no rotation (positions and pair_axis unused).  wire_scales=True
    (hc_append_int4_wire): the bytes that hc_encode_int4 gives for the same rows."""
    return _serve.append_int4(q, k, v, token_rows, codes, scales, positions, table, pair_axis, err, pairing, q_out,
                              stream, wire_scales)


def attend_int4(q, codes, scales, block_tables, q_starts, kv_lens, max_new, workspace, err, causal=True,
                window=0, softmax_scale=None, out=None, lse=None, return_lse=False, stream=None):
    """hc_attend_int4: attention of q [n_tokens, Hq, d] (float16 or bfloat16)
    over the 4-bit cache; returns out, or (out, lse) with return_lse.

    block_tables int32 [n_req, width], q_starts and kv_lens as
    build_block_tables gives them; max_new: at least the largest number of new
    tokens of a request; softmax_scale: 1/sqrt(d) by default.  Rows of tokens that
    belong to no request (a padded step) are not written: in an `out` that the
    call makes, they hold what the memory held."""
    return _serve.attend_int4(q, codes, scales, block_tables, q_starts, kv_lens, max_new, workspace, err, causal,
                              window, softmax_scale, out, lse, return_lse, stream)


def paged_cache(num_slots, H, B, d, dtype=torch.bfloat16, n_layers=None, device="cuda"):
    """Empty K and V pages [num_slots, B, H, d]; with n_layers, one leading dimension more.  dtype: float16 or
    bfloat16, or float32, which append_paged and the codec take but attend_paged refuses."""
    lead = () if n_layers is None else (n_layers,)
    return tuple(torch.zeros(lead + (num_slots, B, H, d), dtype=dtype, device=device) for _ in range(2))


def attend_paged_few_rows(n_req, n_kv_heads, d, table_keys):
    """hc_attend_paged_few_rows: attend_few_rows for attend_paged; table_keys:
    the keys that a row of block_tables has room for."""
    rows = hc.lib().hc_attend_paged_few_rows(n_req, n_kv_heads, d, table_keys)
    if rows < 0:
        hc._check("hc_attend_paged_few_rows", rows)
    return rows


def append_paged(q, k, v, token_rows, k_pages, v_pages, positions, table, pair_axis, err, pairing="half_split",
                 q_out=None, stream=None):
    """hc_append_paged: k, v [n_tokens, H, d] into the pages [num_slots, B, H, d]
    at token_rows (int64), keys rotated; returns the rotated q (None for q
    None).  All of the pages' dtype.  table None: no rotation (positions and
    pair_axis unused)."""
    return _serve.append_paged(q, k, v, token_rows, k_pages, v_pages, positions, table, pair_axis, err, pairing, q_out,
                               stream)


def attend_paged(q, k_pages, v_pages, block_tables, q_starts, kv_lens, max_new, workspace, err, causal=True, window=0,
                 softmax_scale=None, softcap=0.0, slopes=None, positions=None, prefix_lens=None, out=None, lse=None,
                 return_lse=False, stream=None):
    """hc_attend_paged: attention of q [n_tokens, Hq, d] over pages [num_slots,
    B, H, d] of the same dtype (float16 or bfloat16); returns out, or (out, lse)
    with return_lse.

    block_tables, q_starts, kv_lens, max_new, softmax_scale and padded rows as
    for attend_int4.  softcap > 0: scores softcap * tanh(score / softcap).
    slopes (float32 [Hq]): less slope * distance.  positions (int32 [n_tokens],
    not falling within a request): queries at these positions instead of the
    last ones.  prefix_lens (int32 [n_req]): keys that a query sees from before
    them too; a window hides these as it does others (hc_attend_scores)."""
    return _serve.attend_paged(q, k_pages, v_pages, block_tables, q_starts, kv_lens, max_new, workspace, err, causal,
                               window, softmax_scale, softcap, slopes, positions, prefix_lens, out, lse, return_lse,
                               stream)


def merge_attention(out_a, lse_a, out_b, lse_b, out=None, lse=None, stream=None):
    """hc_merge_attention: (out, lse) of the keys of both results; out may be
    out_a or out_b, and lse likewise."""
    return _serve.merge_attention(out_a, lse_a, out_b, lse_b, out, lse, stream)
