"""Long sequences of few heads on the GPU (``-m gpu``): the tensor-core forward
cuts them into pieces, the matrices of one under the chain over the one before.
Against the 64-bit recurrence, at the other tests' bounds."""
import pytest
import torch

import prefix_sum_outer_gb300 as cp
from test_delta_gpu import DEV, DT, args, check, close, f64, make, ref

pytestmark = pytest.mark.gpu


# rows of 64: whole below 64 chunks, then two pieces, three, and six from 192 on
@pytest.mark.parametrize("shape", [
    (1, 2, 1, 64 * 64 - 3, 64, 40, True), (1, 2, 2, 64 * 64 + 1, 128, 64, False),
    (2, 1, 1, 64 * 101, 40, 64, True)], ids=lambda s: "x".join(map(str, s)))
def test_forward_and_backward(shape):
    B, H, Hk, N, D, M, carry = shape
    check(make(B, H, Hk, N, D, M, DT["bf16"], seed=N + D, carry=carry, rate=0.05))


def test_many_pieces():
    x = make(1, 1, 1, 64 * 195 + 17, 64, 64, DT["bf16"], seed=7, carry=True, rate=0.02)
    out, s = cp.causal_product_fwd_delta(*args(x), state_in=x["s0"], return_state=True, scale=0.3)
    r_out, r_s, _ = ref.delta_fwd(*[f64(t) for t in args(x)], 0.3, f64(x["s0"]))
    close(out, r_out, "out")
    close(s, r_s, "state")


def test_pieces_in_a_graph_and_back_to_back():
    """Calls that follow one another on a stream, sharing a workspace, and the
    same call replayed from a graph: the same bits."""
    x = make(2, 4, 2, 64 * 130, 64, 64, DT["bf16"], seed=8, carry=True, rate=0.02)
    B, H, N, M = x["v"].shape
    n = cp.causal_product_delta_workspace_size(B, H, 2, N, 64, M, torch.bfloat16)
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    first, s1 = cp.causal_product_fwd_delta(*args(x), state_in=x["s0"], return_state=True)
    torch.cuda.synchronize()
    out, s = torch.empty_like(first), torch.empty_like(s1)
    call = lambda: cp.causal_product_fwd_delta(*args(x), out=out, workspace=ws, state_in=x["s0"],  # noqa: E731
                                               state_out=s, return_state=True)
    for _ in range(5):
        out.zero_()
        s.zero_()
        for _ in range(3):
            call()
        torch.cuda.synchronize()
        assert torch.equal(out, first) and torch.equal(s, s1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        call()
    for _ in range(5):
        out.zero_()
        s.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first) and torch.equal(s, s1)
    assert cp.causal_product_status(ws) == 0
