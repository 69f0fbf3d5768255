"""The gated delta rule and the q/k norm on the GPU (``-m gpu``) with a stream
named that is not the current one: what a call allocates (results, workspace)
belongs to the stream that it runs on, so that nothing of the current stream's
can still be using it, or get it back too early."""
import pytest
import torch

import prefix_sum_outer_gb300 as cp
import test_qk_rope_gpu as rope
from test_delta_gpu import DT, args, make

pytestmark = pytest.mark.gpu


@pytest.fixture
def allocations(monkeypatch):
    """The streams that were current at every allocation."""
    seen = []
    for name in ("empty", "empty_like", "zeros"):
        real = getattr(torch, name)

        def wrapped(*a, _real=real, **k):
            seen.append(torch.cuda.current_stream().cuda_stream)
            return _real(*a, **k)

        monkeypatch.setattr(torch, name, wrapped)
    return seen


def calls(dt):
    x = make(2, 4, 2, 200, 64, 64, DT[dt], seed=21, carry=True)
    y = rope.make(2, 4, 2, 50, 64, 32, dt, seed=22)
    one = [t[:, :, 0].contiguous() for t in args(x)]

    def run(stream):
        out, s, ckpt = cp.causal_product_fwd_delta(*args(x), state_in=x["s0"], return_state=True,
                                                   save=True, stream=stream)
        got = [out, s, *cp.causal_product_bwd_delta(*args(x), x["go"], ckpt, grad_state_out=x["gs"],
                                                    return_state_grad=True, stream=stream)]
        state = x["s0"].clone()
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        got += [cp.causal_product_decode_delta(*one, state, stream=stream), state]
        w = (y["xq"], y["xk"], y["wq"], y["wk"])
        got += cp.causal_product_qk_rope(*w, y["cos"], y["sin"], stream=stream)
        return got + list(cp.causal_product_qk_rope_bwd(*w, y["gq"], y["gk"], y["cos"], y["sin"],
                                                        stream=stream))
    return run


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_named_stream(dt, allocations):
    run = calls(dt)
    want = run(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    allocations.clear()
    got = run(side)
    assert allocations and set(allocations) == {side.cuda_stream}
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
