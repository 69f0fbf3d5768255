"""The layer norm of nothing (``-m gpu``): a batch of no sequences, like no rows,
gives an empty result, and zero for the weights' gradients."""
import pytest
import torch

import prefix_sum_outer_gb300 as cp
from test_decay_gpu import DEV, DT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("shape,major", [((0, 16), False), ((0, 5, 16), False), ((3, 0, 16), False),
                                         ((0, 2, 5, 16), False), ((0, 2, 5, 16), True),
                                         ((3, 2, 0, 16), True), ((0, 2, 0, 16), False)])
def test_no_rows(dt, shape, major):
    x = torch.empty(shape, dtype=DT[dt], device=DEV, requires_grad=True)
    w, b = (torch.ones(16, dtype=DT[dt], device=DEV, requires_grad=True) for _ in range(2))
    y = cp.layer_norm(x, w, b, token_major=major)
    assert y.shape == ((shape[0], shape[2], shape[1], 16) if major else shape)
    y.sum().backward()
    assert x.grad.shape == x.shape
    assert torch.equal(w.grad, torch.zeros_like(w)) and torch.equal(b.grad, torch.zeros_like(b))
    with torch.no_grad():
        assert cp.layer_norm(x, w, b, token_major=major).shape == y.shape
