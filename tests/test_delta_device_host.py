"""On which device the gated delta rule's and the q/k norm's calls start their
kernels (no GPU needed): the C side launches on the current device, so that has
to be the tensors' when the library is called, and the caller's again after.
The tensors, the CUDA state and the library are stand-ins."""
import types

import pytest
import torch

import prefix_sum_outer_gb300 as cp

B, H, Hk, N, D, M = 2, 4, 2, 5, 16, 16


class Cuda(torch.Tensor):
    """A tensor that says it is on a GPU."""

    index = 1

    def get_device(self):
        return self.index


def tensor(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(Cuda)


@pytest.fixture
def machine(monkeypatch):
    """Two GPUs of which the first is current; what was current at each call."""
    state = types.SimpleNamespace(current=0, at_call=[], streams=[])

    class device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, state.current = state.current, self.index

        def __exit__(self, *a):
            state.current = self.before

    class Library:
        def __getattr__(self, name):
            def call(*a):
                if not name.endswith("_size"):
                    state.at_call.append((name, state.current, a[-1]))
                return 0 if not name.endswith("_size") else 1024
            return call

    monkeypatch.setattr(cp, "load_library", lambda: Library())
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: device(s.device.index))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state.current, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 1000 + i, raising=False)
    monkeypatch.setattr(cp, "_check_device", lambda *ts: None)
    return state


def calls(stream=None):
    qk = [tensor(B, Hk, N, D) for _ in range(2)]
    vo = [tensor(B, H, N, M) for _ in range(2)]
    g = [tensor(B, H, N) for _ in range(2)]
    one = [t[:, :, 0].contiguous() for t in (*qk, vo[0], *g)]
    w = tensor(D)
    yield "causal_product_fwd_delta", lambda: cp.causal_product_fwd_delta(*qk, vo[0], *g, stream=stream)
    yield "causal_product_bwd_delta", lambda: cp.causal_product_bwd_delta(
        *qk, vo[0], *g, vo[1], tensor(4096), stream=stream)
    yield "causal_product_decode_delta", lambda: cp.causal_product_decode_delta(
        *one, tensor(B, H, D, M), stream=stream)
    yield "causal_product_decode_delta", lambda: cp.causal_product_decode_delta(
        *one, tensor(B, H, D, M), out=tensor(B, H, M), stream=stream)
    yield "causal_product_qk_rope", lambda: cp.causal_product_qk_rope(*qk, w, w, stream=stream)
    yield "causal_product_qk_rope_bwd", lambda: cp.causal_product_qk_rope_bwd(
        *qk, w, w, *qk, stream=stream)


@pytest.mark.parametrize("current", [0, 1])
def test_the_tensors_device_is_current_at_the_launch(machine, current):
    machine.current = current
    for name, call in calls():
        call()
        assert machine.at_call == [(name, 1, 1001)]
        assert machine.current == current
        machine.at_call.clear()


def test_a_stream_of_another_device_is_refused(machine):
    stream = types.SimpleNamespace(device=torch.device("cuda", 0), cuda_stream=7)
    for _, call in calls(stream):
        with pytest.raises(RuntimeError):
            call()
    assert not machine.at_call


def test_a_named_stream(machine):
    stream = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=7)
    for name, call in calls(stream):
        call()
        assert machine.at_call == [(name, 1, 1001)] and machine.current == 0
        machine.at_call.clear()
