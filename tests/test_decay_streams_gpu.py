"""Linear attention with a decay and the layer norm on the GPU (``-m gpu``) with a
stream named that is not the current one: what a call allocates (results,
workspace) belongs to the stream that it runs on.  And behind a busy stream, whose
inputs are not there yet when the call is made."""
import pytest
import torch

import prefix_sum_outer_gb300 as cp
from test_decay_gpu import DEV, DT, args, make, results
from test_delta_streams_gpu import allocations  # noqa: F401

pytestmark = pytest.mark.gpu


def calls(dt):
    x = make(2, 4, 2, 500, 64, 64, DT[dt], seed=21, carry=True, lengths=[500, 300])
    one = [t[:, :, 0].contiguous() for t in args(x)[:3]] + [x["g"]]
    w = torch.randn(4, 64, device=DEV).to(DT[dt])

    def run(stream):
        got = list(results(x, stream=stream).values())
        state = x["s0"].clone()
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        got += [cp.causal_product_decode_decay(*one, state, stream=stream), state]
        kw = dict(token_major=True, stream=stream)
        y = cp.causal_product_layer_norm(x["v"], w, w, **kw)
        return got + [y, *cp.causal_product_layer_norm_bwd(x["v"], w, w, y, **kw)]
    return run


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_named_stream(dt, allocations):  # noqa: F811
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


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_behind_a_busy_stream(dt):
    """The calls queue behind long work that makes their inputs; two runs in a row
    whose launches may start under one another's ends."""
    x = make(1, 2, 2, 1500, 64, 128, DT[dt], seed=22, carry=True)
    want = results(x)
    real = {n: t.clone() for n, t in x.items() if t is not None}
    for n in ("q", "k", "v", "go", "s0", "gs"):
        x[n].zero_()
    torch.cuda.synchronize()
    a = torch.randn(8192, 8192, device=DEV, dtype=torch.bfloat16)
    for _ in range(4):
        a = (a @ a).clamp(-1, 1)
    for n in ("q", "k", "v", "go", "s0", "gs"):
        x[n].copy_(real[n])
    first, second = results(x), results(x)
    torch.cuda.synchronize()
    for n, t in want.items():
        assert torch.equal(first[n], t) and torch.equal(second[n], t)


def test_workspace_of_the_caller():
    """Too small, misplaced or with gaps: refused; float32 of as many bytes: taken."""
    x = make(1, 2, 1, 700, 64, 64, torch.bfloat16, seed=23)
    w = torch.ones(64, device=DEV, dtype=torch.bfloat16)
    sizes = [cp.causal_product_decay_workspace_size(1, 2, 1, 700, 64, 64, torch.bfloat16, b)
             for b in (False, True)]
    sizes.append(cp.load_library().causal_product_layer_norm_workspace_size(1, 2, 700, 64, 1))
    for n, call in zip(sizes, (
            lambda ws: cp.causal_product_fwd_decay(*args(x), workspace=ws),
            lambda ws: cp.causal_product_bwd_decay(*args(x), x["go"], workspace=ws),
            lambda ws: cp.causal_product_layer_norm_bwd(x["v"], w, w, x["go"], workspace=ws))):
        want = call(None)
        for bad in (torch.zeros(n, dtype=torch.uint8), torch.zeros(n, dtype=torch.uint8).pin_memory()):
            with pytest.raises(RuntimeError):
                call(bad)
        with pytest.raises(ValueError):
            call(torch.zeros(2 * n, dtype=torch.uint8, device=DEV)[::2])
        with pytest.raises(cp.CausalProductError):
            call(torch.zeros(n // 4 - 1, device=DEV))
        got = call(torch.zeros((n + 3) // 4, device=DEV))
        torch.cuda.synchronize()
        for a, b in zip((got,) if torch.is_tensor(got) else got,
                        (want,) if torch.is_tensor(want) else want):
            assert torch.equal(a, b)
