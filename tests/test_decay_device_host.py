"""On which device the calls of linear attention with a decay for each head and
of the layer norm start their kernels (no GPU needed): the C side launches on the
current device, so that has to be the tensors' when the library is called, and
the caller's again after.  The tensors, the CUDA state and the library are
stand-ins."""
import types

import pytest
import torch

import prefix_sum_outer_gb300 as cp
from test_delta_device_host import machine, tensor  # noqa: F401

B, H, Hk, N, D, M = 2, 4, 2, 5, 16, 16


def calls(stream=None):
    qk = [tensor(B, Hk, N, D) for _ in range(2)]
    v, go, g = tensor(B, H, N, M), tensor(B, H, N, M), tensor(H)
    n = tensor(B, dtype=torch.int32)
    one = [t[:, :, 0].contiguous() for t in (*qk, v)]
    w = tensor(M)
    kw = dict(stream=stream, lengths=n)
    yield "causal_product_fwd_decay", lambda: cp.causal_product_fwd_decay(*qk, v, g, **kw)
    yield "causal_product_bwd_decay", lambda: cp.causal_product_bwd_decay(*qk, v, g, go, **kw)
    yield "causal_product_decode_decay", lambda: cp.causal_product_decode_decay(
        *one, g, tensor(B, H, D, M), stream=stream)
    yield "causal_product_layer_norm", lambda: cp.causal_product_layer_norm(
        v, w, w, token_major=True, stream=stream)
    yield "causal_product_layer_norm_bwd", lambda: cp.causal_product_layer_norm_bwd(
        v, w, w, go, stream=stream)


@pytest.mark.parametrize("current", [0, 1])
def test_the_tensors_device_is_current_at_the_launch(machine, current):  # noqa: F811
    machine.current = current
    for name, call in calls():
        call()
        assert machine.at_call == [(name, 1, 1001)]
        assert machine.current == current
        machine.at_call.clear()


def test_a_stream_of_another_device_is_refused(machine):  # noqa: F811
    stream = types.SimpleNamespace(device=torch.device("cuda", 0), cuda_stream=7)
    for _, call in calls(stream):
        with pytest.raises(RuntimeError):
            call()
    assert not machine.at_call


def test_a_named_stream(machine):  # noqa: F811
    stream = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=7)
    for name, call in calls(stream):
        call()
        assert machine.at_call == [(name, 1, 1001)] and machine.current == 0
        machine.at_call.clear()
