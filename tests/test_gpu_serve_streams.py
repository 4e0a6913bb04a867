"""The serving calls on a stream of the caller's: what they allocate belongs to that stream."""
import pytest

from tests.test_gpu_serve import serve, workspace  # noqa: F401
from tests.test_gpu_serve_refusals import args  # noqa: F401

pytestmark = pytest.mark.gpu


def _owner(tensor):
    """The stream whose memory the tensor lies in."""
    import torch
    for segment in torch.cuda.memory_snapshot():
        if segment["address"] <= tensor.data_ptr() < segment["address"] + segment["total_size"]:
            return segment["stream"]
    raise AssertionError("not in any segment")


def _made(call, result):
    return list(result) if call in ("build_block_tables", "attend_int4") else [result]


@pytest.mark.parametrize("call", ["build_block_tables", "rope_axes", "append_int4", "attend_int4"])
def test_outputs_are_allocated_on_the_calls_stream(serve, args, call):  # noqa: F811
    import torch
    kw = dict(args[call])
    if call == "attend_int4":
        kw["return_lse"] = True
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = [t.clone() for t in _made(call, getattr(serve, call)(**kw))]
    torch.cuda.synchronize()
    for stream, owner in ((side, side.cuda_stream), (side.cuda_stream, side.cuda_stream), (0, 0), (1, 0), (None, 0)):
        got = _made(call, getattr(serve, call)(**kw, stream=stream))
        torch.cuda.synchronize()
        assert all(_owner(t) == owner for t in got)
        if call != "build_block_tables":        # which has taken its slots by now
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(side):
        got = _made(call, getattr(serve, call)(**kw))
    torch.cuda.synchronize()
    assert all(_owner(t) == side.cuda_stream for t in got)
    assert torch.cuda.current_stream().cuda_stream == 0         # as it was
    with pytest.raises(ValueError):              # cudaStreamPerThread
        getattr(serve, call)(**kw, stream=2)


def test_a_per_thread_stream_takes_outputs_that_are_given(serve, args):  # noqa: F811
    import torch
    kw = args["rope_axes"]
    want = serve.rope_axes(**kw)
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    serve.rope_axes(**kw, out=out, stream=2)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_a_block_that_queued_work_still_writes(serve):  # noqa: F811
    """A tensor freed on the current stream with its write still to come; a call of the same size on another stream."""
    import torch
    x = torch.randn(300, 4, 64, device="cuda")
    pos = torch.arange(300, dtype=torch.int32, device="cuda")
    table, err = serve.rotation_table(300, 32, 1e4), torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda **kw: serve.rope_axes(x, pos, table, (0,) * 32, err, **kw)
    want = call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = torch.empty_like(x)
    torch.cuda._sleep(100_000_000)
    freed.fill_(7.0)
    del freed
    got = call(stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and int(err) == 0
