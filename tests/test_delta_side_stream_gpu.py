"""Calls with a stream named, as a user meets them (``-m gpu``): the stream is
busy when the call is made, the call returns at once, and the current stream
goes on allocating and writing.  What the call allocated must not come back to
the current stream before its kernels have run."""
import pytest
import torch

from test_delta_streams_gpu import calls

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_memory_of_a_call_on_a_busy_stream(dt):
    run = calls(dt)
    want = run(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    run(side)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)   # about a tenth of a second
    got = run(side)
    assert not side.query()              # nothing of it has run yet
    # every size that the calls may have left behind, overwritten at once
    held = [torch.full((1 << n,), float("nan"), device="cuda") for n in range(6, 24) for _ in range(8)]
    torch.cuda.current_stream().synchronize()
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert len(held) == 18 * 8
