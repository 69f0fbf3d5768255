"""The layer norm's backward with one or both weights' gradients left out (``-m
gpu``): the others keep their bits."""
import pytest
import torch

import prefix_sum_outer_gb300 as cp
from test_decay_gpu import DEV, DT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lead,C,major", [((2, 4, 70), 64, True), ((300,), 33, False), ((3, 50), 1024, False),
                                          ((20,), 16384, False)])
def test_the_others_keep_their_bits(dt, lead, C, major):
    gen = torch.Generator(device=DEV).manual_seed(C)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV).to(DT[dt])  # noqa: E731
    x, w, b = rnd(*lead, C), rnd(C), rnd(C)
    gy = rnd(*((lead[0], lead[2], lead[1]) if major else lead), C)
    call = lambda **kw: cp.causal_product_layer_norm_bwd(x, w, b, gy, token_major=major, **kw)  # noqa: E731
    want = call()
    for weight, bias in ((False, False), (True, False), (False, True)):
        got = call(weight_grad=weight, bias_grad=bias)
        assert torch.equal(got[0], want[0])
        assert torch.equal(got[1], want[1]) if weight else got[1] is None
        assert torch.equal(got[2], want[2]) if bias else got[2] is None
    # with neither there is nothing to gather: a workspace of 256 bytes is enough
    small = torch.empty(256, dtype=torch.uint8, device=DEV)
    assert torch.equal(call(weight_grad=False, bias_grad=False, workspace=small)[0], want[0])
    with pytest.raises(cp.CausalProductError):
        call(workspace=small)
    # frozen weights by autograd
    leaf = x.clone().requires_grad_(True)
    cp.layer_norm(leaf, w, b, token_major=major).backward(gy)
    assert torch.equal(leaf.grad, want[0])
