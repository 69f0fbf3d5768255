"""The q/k norm with rotation on the GPU (``-m gpu``) where a feature that is not
turned is infinite: the rotation pairs features (i, i + R/2), i < R/2, alone, so
what stands still reaches no other feature."""
import pytest
import torch

import prefix_sum_outer_gb300 as cp
import test_qk_rope_gpu as rope
from test_delta_gpu import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,R,f", [(64, 16, 20), (64, 16, 60), (128, 64, 100), (96, 32, 40), (64, 0, 5),
                                   (72, 24, 30), (40, 8, 39)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_infinite_weight_and_gradient(D, R, f, dt):
    x = rope.make(2, 3, 1, 11, D, R, dt, seed=D + f)
    kw = dict(cos=x["cos"], sin=x["sin"])
    there = torch.zeros(D, dtype=torch.bool, device=DEV)
    there[f] = True
    w = x["wq"].clone()
    w[f] = float("inf")
    q, _ = cp.causal_product_qk_rope(x["xq"], x["xk"], w, x["wk"], **kw)
    assert torch.equal(torch.isfinite(q).all(0).all(0).all(0), ~there)
    gq = x["gq"].clone()
    gq[1, 2, 7, f] = float("inf")
    dx, _, dw, _ = cp.causal_product_qk_rope_bwd(x["xq"], x["xk"], x["wq"], x["wk"], gq, x["gk"], **kw)
    assert torch.equal(torch.isfinite(dw), ~there)
    rows = torch.ones(dx.shape[:3], dtype=torch.bool, device=DEV)
    rows[1, 2, 7] = False
    assert torch.isfinite(dx[rows]).all()
