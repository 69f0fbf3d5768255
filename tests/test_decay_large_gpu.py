"""Linear attention with a decay and the layer norm on tensors of more than 2^31
elements (``-m gpu``).  The state forgets within a few hundred rows (e^-0.1 a
row), so the last rows of a long sequence are those of its end alone."""
import pytest
import torch

import prefix_sum_outer_gb300 as cp
from test_decay_gpu import DEV

pytestmark = pytest.mark.gpu

N, END = (1 << 23) + 128, 2048


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("D,M,dtype", [(128, 8, torch.bfloat16), (8, 128, torch.bfloat16),
                                       (128, 8, torch.float32)], ids=str)
def test_forward_and_backward(D, M, dtype):
    gen = torch.Generator(device=DEV).manual_seed(D + M)
    rnd = lambda n: torch.randn((1, 2, N, n), generator=gen, device=DEV, dtype=dtype)  # noqa: E731
    x = [rnd(D), rnd(D), rnd(M)]
    g, go = torch.full((2,), -0.1, device=DEV), rnd(M)
    assert x[0].numel() > 2 ** 31 or x[2].numel() > 2 ** 31

    def run(cut):
        y = [t[:, :, cut].contiguous() for t in (*x, go)] if cut is not None else [*x, go]
        out, s = cp.causal_product_fwd_decay(*y[:3], g, return_state=True)
        return (out, *cp.causal_product_bwd_decay(*y[:3], g, y[3])), s

    got, s = run(None)
    # rows of the end, from a state that the rows before it made (all but forgotten)
    end, e_s = run(slice(N - 2 * END, None))
    for a, b in zip(got, end):
        a, b = a[:, :, N - END:].double(), b[:, :, END:].double()
        assert (a - b).norm() <= 1e-4 * b.norm()
    assert (s - e_s).norm() <= 1e-6 * e_s.norm()
    # and of the beginning, whose gradients no later row reaches
    begin, _ = run(slice(0, 2 * END))
    for a, b in zip(got, begin):
        a, b = a[:, :, :END].double(), b[:, :, :END].double()
        assert (a - b).norm() <= 1e-4 * b.norm()


def test_norm():
    B, H, n, C = 1, 17, (1 << 20) + 7, 128
    gen = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn((B, H, n, C), generator=gen, device=DEV, dtype=torch.bfloat16)
    w = torch.randn((H, C), generator=gen, device=DEV, dtype=torch.bfloat16)
    assert x.numel() > 2 ** 31
    y = cp.causal_product_layer_norm(x, w, w, token_major=True)
    dx = cp.causal_product_layer_norm_bwd(x, w, w, y, token_major=True)[0]
    lo = n - 500
    z = cp.causal_product_layer_norm(x[:, :, lo:], w, w, token_major=True)
    dz = cp.causal_product_layer_norm_bwd(x[:, :, lo:], w, w, z, token_major=True)[0]
    assert torch.equal(y[:, lo:], z) and torch.equal(dx[:, :, lo:], dz)
