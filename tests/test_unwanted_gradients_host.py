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


@pytest.mark.parametrize("x_grad,w_grad,b_grad", [(True, False, False), (True, True, False),
                                                  (False, False, True), (True, True, True)])
def test_the_weights_of_a_layer_norm(monkeypatch, x_grad, w_grad, b_grad):
    """Frozen weights have no sums to gather."""
    seen = []

    def bwd(x, w, b, gy, *a, weight_grad=True, bias_grad=True, **kw):
        seen.append((weight_grad, bias_grad))
        return (torch.zeros_like(x), torch.zeros_like(w) if weight_grad else None,
                torch.zeros_like(b) if bias_grad else None)

    monkeypatch.setattr(cp, "causal_product_layer_norm_bwd", bwd)
    monkeypatch.setattr(cp, "causal_product_layer_norm", lambda x, *a, **kw: x.clone())
    x, w, b = (torch.ones(s).requires_grad_(g) for s, g in (((3, 8), x_grad), ((8,), w_grad),
                                                            ((8,), b_grad)))
    cp.layer_norm(x, w, b).sum().backward()
    assert seen == [(w_grad, b_grad)]
    assert (w.grad is not None, b.grad is not None) == (w_grad, b_grad)
