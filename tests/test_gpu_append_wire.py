"""Appended rows as the encoder's bytes: hc_append_int4_wire against hc_encode_int4 of the same rows."""
import pytest

from tests.serve_cases import DT
from tests.test_gpu_serve import _err, serve  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", ["f16", "f32"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("H,B,d,group", [(4, 16, 128, 32), (3, 32, 64, 64), (2, 64, 128, 128), (5, 16, 64, 32)])
@pytest.mark.parametrize("size", [1.0, 3e-3, 2e3])
def test_append_gives_the_encoders_bytes(serve, scale, dtype, H, B, d, group, size):  # noqa: F811
    import torch
    from kv_cache_quantization_hc_gb300 import hc
    S = 40
    g = torch.Generator(device="cuda")
    g.manual_seed(d + group)
    pool = (torch.randn(2, S, B, H, d, device="cuda", generator=g) * size).to(getattr(torch, DT[dtype]))
    pool[:, 0, 0] = 0                                             # scales of 0
    pool[:, 1, :, :, ::2] = pool[:, 1].abs().amax(-1, keepdim=True) / 2   # halves of the largest: quotients near 3.5
    wire_c, wire_s = serve.int4_cache(S, H, B, d, group, scale)
    err = _err()
    order = torch.arange(S, dtype=torch.int32, device="cuda")
    hc.hc_encode_int4(pool[0], pool[1], hc.paged_desc(pool[0]), order, None, S, group, hc.DTYPE_NAMES[scale], wire_c, wire_s,
                      err)
    codes, scales = serve.int4_cache(S, H, B, d, group, scale)
    serve.append_int4(None, pool[0].view(S * B, H, d), pool[1].view(S * B, H, d), torch.arange(S * B, device="cuda"),
                      codes, scales, None, None, None, err, wire_scales=True)
    assert int(err) == 0 and torch.equal(codes, wire_c) and torch.equal(scales, wire_s)


@pytest.mark.parametrize("pairing,rot", [("half_split", 128), ("interleaved", 128), ("half_split", 96)])
def test_rotated_keys_too(serve, pairing, rot):  # noqa: F811
    """Keys turned in fp32 by hc_rope_axes and encoded, against keys turned by the append."""
    import torch
    from kv_cache_quantization_hc_gb300 import hc
    S, B, H, d, group = 30, 16, 8, 128, 32
    g = torch.Generator(device="cuda")
    g.manual_seed(rot)
    k, v = (torch.randn(S * B, H, d, device="cuda", generator=g) for _ in range(2))
    pos = torch.arange(S * B, dtype=torch.int32, device="cuda")
    table, axes, err = serve.rotation_table(S * B, rot // 2, 1e4), (0,) * (rot // 2), _err()
    turned = serve.rope_axes(k, pos, table, axes, err, pairing=pairing)
    pool = torch.stack([turned, v]).view(2, S, B, H, d)
    wire_c, wire_s = serve.int4_cache(S, H, B, d, group, "f32")
    hc.hc_encode_int4(pool[0], pool[1], hc.paged_desc(pool[0]), torch.arange(S, dtype=torch.int32, device="cuda"), None, S, group,
                      hc.HC_F32, wire_c, wire_s, err)
    codes, scales = serve.int4_cache(S, H, B, d, group, "f32")
    serve.append_int4(None, k, v, torch.arange(S * B, device="cuda"), codes, scales, pos, table, axes, err, pairing=pairing,
                      wire_scales=True)
    assert int(err) == 0 and torch.equal(codes, wire_c) and torch.equal(scales, wire_s)
