"""Serving from the 4-bit cache: the calls of include/hc.h on torch tensors.

A layer's cache is an INT4 wire over its slots, codes [num_slots, 2, H, B,
d/2] and scales [num_slots, 2, H, B, d/group] (`int4_cache` makes one; the
codes and scales of hc_encode_int4 with one layer are one too).  One step of
a decoder:

  step = build_block_tables(cached_lens, new_lens, free_slots, tables, B, n_tokens, err)
  per layer:
    q = append_int4(q, k, v, step.token_rows, codes, scales, positions, table, pair_axis, err)
    o = attend_int4(q, codes, scales, tables, step.q_starts, step.kv_lens, max_new, workspace, err)

Every call takes its tensors on the GPU, enqueues its kernel on `stream`
(default: torch's current stream) and returns without synchronising; an
argument it cannot take raises.  What only the device sees (a slot, length or
position out of range) sets bits HC_DEVERR_* in `err`, an int32 tensor that
the caller zeroes and reads.  Tensors used on another stream than the one
they were allocated on are the caller's to record (`Tensor.record_stream`).
"""
import ctypes
from collections import namedtuple

import torch

from . import hc

StepTables = namedtuple("StepTables", "q_starts kv_lens token_req token_pos token_rows n_taken")
StepTables.__doc__ = """Addressing of one step, as hc_build_block_tables defines it: q_starts
int32 [n_req + 1], kv_lens int32 [n_req], token_req and token_pos int32
[n_tokens], token_rows int64 [n_tokens], n_taken int32 [1]."""

_DTYPES = {torch.float32: hc.HC_F32, torch.float16: hc.HC_F16, torch.bfloat16: hc.HC_BF16}


def _device(x, name, dtype, numel=None):
    """Address of a contiguous CUDA tensor of `dtype` with at least `numel` elements."""
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if x.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {x.dtype}")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and x.numel() < numel:
        raise ValueError(f"{name} has {x.numel()} elements; the call addresses {numel}")
    return x.data_ptr()


def _rows(x, name, heads, d, dtype=None, n=None):
    """hc_rows of a tensor [n_tokens, heads, d] whose channels are adjacent."""
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if x.dim() != 3 or (heads is not None and x.shape[1] != heads) or (d is not None and x.shape[2] != d):
        raise ValueError(f"{name} must be [n_tokens, {heads}, {d}], not {tuple(x.shape)}")
    if dtype is not None and x.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {x.dtype}")
    if n is not None and x.shape[0] != n:
        raise ValueError(f"{name} has {x.shape[0]} tokens, not {n}")
    st, sh, sc = x.stride()
    if sc != 1 and x.shape[2] != 1:
        raise ValueError(f"the channels of {name} must be adjacent")
    return hc.hc_rows(x.data_ptr(), st, sh)


def _cache_desc(codes, scales):
    """hc_int4_cache of a layer's codes and scales, their shapes checked."""
    if codes.dim() != 5 or scales.dim() != 5 or codes.shape[1] != 2 or codes.shape[:4] != scales.shape[:4]:
        raise ValueError("codes must be [num_slots, 2, H, B, d/2] and scales [num_slots, 2, H, B, d/group]")
    S, _, H, B, half = codes.shape
    d, groups = 2 * half, scales.shape[4]
    if groups < 1 or d % groups:
        raise ValueError(f"scales hold {groups} groups per row of {d} channels")
    if scales.dtype not in (torch.float16, torch.float32):
        raise ValueError(f"scales must be float16 or float32, not {scales.dtype}")
    _device(codes, "codes", torch.uint8)
    _device(scales, "scales", scales.dtype)
    return hc.hc_int4_cache(H, d, B, S, d // groups, _DTYPES[scales.dtype])


_ROPE_AXES = {}


def _pair_axis(pair_axis):
    """The axes of the pairs as the C array, made once per distinct tuple."""
    key = tuple(pair_axis)
    if key not in _ROPE_AXES:
        if not 1 <= len(key) <= 128 or any(not 0 <= a < 8 for a in key):
            raise ValueError("pair_axis holds the axis (0..7) of each of 1 to 128 pairs")
        _ROPE_AXES[key] = (ctypes.c_uint8 * 128)(*key)
    return _ROPE_AXES[key], len(key)


def _rope_desc(positions, table, pair_axis, pairing, inverse, n):
    if positions.dim() == 1:
        positions = positions.unsqueeze(0)
    if positions.dim() != 2 or positions.shape[1] != n or not positions.is_cuda:
        raise ValueError(f"positions must be a CUDA tensor [n_axes, {n}]")
    if positions.dtype != torch.int32 or (n > 1 and positions.stride(1) != 1):
        raise ValueError("positions must be int32, each axis's adjacent")
    axes, half = _pair_axis(pair_axis)
    if table.dim() != 3 or table.shape[1] != half or table.shape[2] != 2:
        raise ValueError(f"table must be [n_positions, {half}, 2]")
    n_axes = positions.shape[0]
    stride = positions.stride(0) if n_axes > 1 else 0
    return hc.hc_rope_axes_desc(positions.data_ptr(), stride, _device(table, "table", torch.float32), n_axes,
                                table.shape[0], 2 * half, hc.PAIRING_NAMES[pairing], int(inverse), axes)


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
    """A workspace for attend_int4 (zeroed; each call leaves it ready for the next).
    Calls that may run at the same time need one each."""
    return torch.zeros(hc.lib().hc_attend_int4_workspace(), dtype=torch.uint8, device=device)


def build_block_tables(cached_lens, new_lens, free_slots, block_tables, block_size, n_tokens, err,
                       out=None, stream=None):
    """hc_build_block_tables: writes the new blocks' slots into block_tables
    (int32 [n_req, width], updated in place) and returns the StepTables
    (`out`: one to write into, its token arrays of n_tokens entries)."""
    n_req = cached_lens.numel()
    dev = cached_lens.device
    if block_tables.dim() != 2 or block_tables.shape[0] != n_req or block_tables.dtype != torch.int32 \
            or not block_tables.is_cuda or (block_tables.shape[1] > 1 and block_tables.stride(1) != 1):
        raise ValueError(f"block_tables must be int32 [{n_req}, width] on the GPU, each row adjacent")
    if out is None:
        i32 = torch.empty(2 * n_req + 2 + 2 * n_tokens, dtype=torch.int32, device=dev)
        # token arrays first: 16-byte aligned where n_tokens is a multiple of 4
        req, pos, starts, kv, taken = i32.split([n_tokens, n_tokens, n_req + 1, n_req, 1])
        out = StepTables(starts, kv, req, pos, torch.empty(n_tokens, dtype=torch.int64, device=dev), taken)
    stride = block_tables.stride(0) if n_req > 1 else block_tables.shape[1]
    hc._check("hc_build_block_tables", hc.lib().hc_build_block_tables(
        _device(cached_lens, "cached_lens", torch.int32), _device(new_lens, "new_lens", torch.int32, n_req),
        n_req, block_size, _device(free_slots, "free_slots", torch.int32), free_slots.numel(),
        block_tables.data_ptr(), stride, block_tables.shape[1], n_tokens,
        _device(out.q_starts, "q_starts", torch.int32, n_req + 1),
        _device(out.kv_lens, "kv_lens", torch.int32, n_req),
        _device(out.token_req, "token_req", torch.int32, n_tokens),
        _device(out.token_pos, "token_pos", torch.int32, n_tokens),
        _device(out.token_rows, "token_rows", torch.int64, n_tokens),
        _device(out.n_taken, "n_taken", torch.int32, 1), _device(err, "err", torch.int32, 1),
        hc._stream(stream)))
    return out


def rope_axes(x, positions, table, pair_axis, err, pairing="half_split", inverse=False, out=None,
              stream=None):
    """hc_rope_axes: x [n_tokens, n_heads, d] with its pairs turned.

    positions int32 [n_axes, n_tokens]; table [n_positions, pairs, 2]; pair_axis:
    the axis of each pair.  inverse=True turns back, which is also the gradient
    of the rotation.  out=x rotates in place; queries and keys that lie in one
    packed buffer are one call on the view of both."""
    n, heads, d = x.shape
    y = torch.empty((n, heads, d), dtype=x.dtype, device=x.device) if out is None else out
    hc._check("hc_rope_axes", hc.lib().hc_rope_axes(
        _rows(x, "x", None, None), _rows(y, "out", heads, d, x.dtype, n), _DTYPES[x.dtype], n, heads, d,
        _rope_desc(positions, table, pair_axis, pairing, inverse, n), _device(err, "err", torch.int32, 1),
        hc._stream(stream)))
    return y


def append_int4(q, k, v, token_rows, codes, scales, positions, table, pair_axis, err,
                pairing="half_split", q_out=None, stream=None):
    """hc_append_int4: k, v [n_tokens, H, d] into the cache at token_rows
    (int64), keys rotated; returns the rotated q (None for q None).  table
    None: no rotation (positions and pair_axis unused)."""
    desc = _cache_desc(codes, scales)
    n, H, d = k.shape[0], desc.n_kv_heads, desc.d_head
    if k.dtype not in _DTYPES:
        raise ValueError(f"k must be float32, float16 or bfloat16, not {k.dtype}")
    heads, qr, qo = 0, None, None
    if q is not None:
        heads = q.shape[1]
        qr = _rows(q, "q", heads, d, k.dtype, n)
        q_out = torch.empty((n, heads, d), dtype=q.dtype, device=q.device) if q_out is None else q_out
        qo = _rows(q_out, "q_out", heads, d, k.dtype, n)
    rope = None if table is None else _rope_desc(positions, table, pair_axis, pairing, False, n)
    hc._check("hc_append_int4", hc.lib().hc_append_int4(
        qr, _rows(k, "k", H, d), _rows(v, "v", H, d, k.dtype, n), _DTYPES[k.dtype], n, heads, rope,
        _device(token_rows, "token_rows", torch.int64, n), desc, codes.data_ptr(), scales.data_ptr(), qo,
        _device(err, "err", torch.int32, 1), hc._stream(stream)))
    return q_out


def attend_int4(q, codes, scales, block_tables, q_starts, kv_lens, max_new, workspace, err, causal=True,
                window=0, softmax_scale=None, out=None, lse=None, return_lse=False, stream=None):
    """hc_attend_int4: attention of q [n_tokens, Hq, d] (float16 or bfloat16)
    over the 4-bit cache; returns out, or (out, lse) with return_lse.

    block_tables int32 [n_req, width], q_starts and kv_lens as
    build_block_tables gives them; max_new: at least the largest number of new
    tokens of a request; softmax_scale: 1/sqrt(d) by default."""
    desc = _cache_desc(codes, scales)
    n, heads, d = q.shape
    if q.dtype not in _DTYPES:
        raise ValueError(f"q must be float16 or bfloat16, not {q.dtype}")
    n_req = kv_lens.numel()
    if block_tables.dim() != 2 or block_tables.shape[0] != n_req or block_tables.dtype != torch.int32 \
            or not block_tables.is_cuda or (block_tables.shape[1] > 1 and block_tables.stride(1) != 1):
        raise ValueError(f"block_tables must be int32 [{n_req}, width] on the GPU, each row adjacent")
    y = torch.empty((n, heads, d), dtype=q.dtype, device=q.device) if out is None else out
    if return_lse and lse is None:
        lse = torch.empty((n, heads), dtype=torch.float32, device=q.device)
    stride = block_tables.stride(0) if n_req > 1 else block_tables.shape[1]
    hc._check("hc_attend_int4", hc.lib().hc_attend_int4(
        _rows(q, "q", None, desc.d_head), _rows(y, "out", heads, d, q.dtype, n),
        None if lse is None else _device(lse, "lse", torch.float32, n * heads), _DTYPES[q.dtype], n, heads,
        desc, codes.data_ptr(), scales.data_ptr(), block_tables.data_ptr(), stride, block_tables.shape[1],
        _device(q_starts, "q_starts", torch.int32, n_req + 1), _device(kv_lens, "kv_lens", torch.int32),
        n_req, max_new, int(causal), window, d ** -0.5 if softmax_scale is None else softmax_scale,
        _device(workspace, "workspace", torch.uint8), workspace.numel(), _device(err, "err", torch.int32, 1),
        hc._stream(stream)))
    return (y, lse) if return_lse else y
