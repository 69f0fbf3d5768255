"""Autograd around linear attention with a decay and the layer norm (``-m gpu``): a
gradient asked for changes no result, and a second derivative, which neither has,
is refused rather than left out."""
import pytest
import torch

import prefix_sum_outer_gb300 as cp
from test_decay_gpu import DEV, DT, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("return_state", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_results_with_and_without_gradients(dt, return_state):
    x = make(2, 4, 2, 700, 64, 64, DT[dt], seed=31, carry=True, lengths=[700, 333])
    rows = [x[n].clone().requires_grad_(True) for n in ("q", "k", "v")]
    call = lambda: cp.causal_product_decay(*rows, x["g"], state=x["s0"], scale=0.3,  # noqa: E731
                                           lengths=x["n"], return_state=return_state)
    with_grad = call()
    with torch.no_grad():
        without = call()
    pairs = zip(with_grad, without) if return_state else [(with_grad, without)]
    for a, b in pairs:
        assert a.requires_grad and not b.requires_grad
        assert torch.equal(a.detach(), b)
    w = torch.randn(4, 64, device=DEV).to(DT[dt]).requires_grad_(True)
    y = cp.layer_norm(x["v"], w, token_major=True)
    with torch.no_grad():
        z = cp.layer_norm(x["v"], w, token_major=True)
    assert y.requires_grad and not z.requires_grad
    assert torch.equal(y.detach(), z)


def test_second_derivatives_are_refused():
    x = make(1, 2, 2, 70, 16, 16, torch.float32, seed=32)
    q, k, v = (x[n].clone().requires_grad_(True) for n in ("q", "k", "v"))
    (dv,) = torch.autograd.grad(cp.causal_product_decay(q, k, v, x["g"]).square().sum(), v,
                                create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(dv.sum(), q)
    (dv,) = torch.autograd.grad(cp.layer_norm(v).square().sum(), v, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(dv.sum(), v)
