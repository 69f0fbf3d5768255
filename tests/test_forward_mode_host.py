"""Forward-mode derivatives, which no operator here has, are refused and not left
out (no GPU needed; the C calls are stand-ins)."""
import pytest
import torch
from torch.autograd import forward_ad

import prefix_sum_outer_gb300 as cp

q, v, g = torch.ones(1, 2, 3, 8), torch.ones(1, 2, 3, 8), torch.zeros(2)
s, beta = torch.ones(1, 2, 8, 8), torch.ones(1, 2, 3)
x, w = torch.ones(3, 8), torch.ones(8)

# the operators, and the arguments that may carry a tangent
CALLS = {
    "layer_norm": (lambda *a: cp.layer_norm(*a), (x, w, w)),
    "causal_product_decay": (lambda q, k, v, g, s: cp.causal_product_decay(q, k, v, g, state=s),
                             (q, q, v, g, s)),
    "causal_product_delta": (lambda q, k, v, g, b, s: cp.causal_product_delta(q, k, v, g, b, state=s),
                             (q, q, v, beta - 1, beta, s)),
}


@pytest.fixture(autouse=True)
def stand_ins(monkeypatch):
    monkeypatch.setattr(cp, "causal_product_layer_norm", lambda x, *a, **k: x.detach().clone())
    for name in ("causal_product_fwd_decay", "causal_product_fwd_delta"):
        monkeypatch.setattr(cp, name, lambda q, k, v, *a, **kw: v.detach().clone())


@pytest.mark.parametrize("name", CALLS)
def test_a_tangent_is_refused(name):
    call, args = CALLS[name]
    assert call(*args).shape == args[2 if len(args) > 3 else 0].shape
    for i in range(len(args)):
        with forward_ad.dual_level():
            dual = [forward_ad.make_dual(t, torch.ones_like(t)) if j == i else t
                    for j, t in enumerate(args)]
            with pytest.raises(NotImplementedError):
                call(*dual)
            with torch.no_grad(), pytest.raises(NotImplementedError):
                call(*dual)
            call(*args)  # the others' values are nobody's tangent


def test_through_the_function_transforms():
    with pytest.raises(NotImplementedError):
        torch.func.jvp(lambda t: cp.layer_norm(t), (x,), (x,))
