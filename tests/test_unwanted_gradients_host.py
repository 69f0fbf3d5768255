"""What the autograd wrappers ask of the C calls: the gradients that somebody
wants (no GPU needed; the C calls are stand-ins)."""
import pytest
import torch

import prefix_sum_outer_gb300 as cp


@pytest.fixture
def asked(monkeypatch):
    seen = []

    def bwd_decay(q, k, v, g, go, state_in=None, return_state_grad=False, **kw):
        seen.append(return_state_grad)
        got = (torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v))
        return got + ((torch.zeros_like(state_in),) if return_state_grad else ())

    monkeypatch.setattr(cp, "causal_product_bwd_decay", bwd_decay)
    monkeypatch.setattr(cp, "causal_product_fwd_decay", lambda q, k, v, *a, **kw: v.clone())
    return seen


@pytest.mark.parametrize("wanted", [False, True])
def test_the_state_of_a_decay(asked, wanted):
    """A carried state that is a constant (truncated backpropagation) has no
    gradient to compute."""
    q, s = torch.ones(1, 2, 3, 8), torch.ones(1, 2, 8, 8).requires_grad_(wanted)
    v = torch.ones(1, 2, 3, 8).requires_grad_(True)
    cp.causal_product_decay(q, q, v, torch.zeros(2), state=s).sum().backward()
    assert asked == [wanted]
    assert v.grad is not None and (s.grad is not None) == wanted
