"""The gated delta rule and the q/k norm on tensors of more than 2^31 elements
(``-m gpu``).  The state forgets within a few hundred rows (e^-0.1 a row), so the
last rows of a long sequence are those of its end alone."""
import pytest
import torch

import prefix_sum_outer_gb300 as cp
from test_delta_gpu import DEV

pytestmark = pytest.mark.gpu

N, END = (1 << 23) + 128, 2048


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def inputs(D, M, dtype):
    gen = torch.Generator(device=DEV).manual_seed(D + M)
    rnd = lambda n: torch.randn((1, 2, N, n), generator=gen, device=DEV, dtype=dtype)  # noqa: E731
    q, k = rnd(D), rnd(D)
    q *= D ** -0.5
    k *= D ** -0.5
    g = torch.full((1, 2, N), -0.1, device=DEV)
    return q, k, rnd(M), g, torch.rand((1, 2, N), generator=gen, device=DEV), rnd(M)


@pytest.mark.parametrize("D,M,dtype", [(128, 8, torch.bfloat16), (8, 128, torch.bfloat16),
                                       (128, 8, torch.float32)], ids=str)
def test_forward_and_backward(D, M, dtype):
    *x, go = inputs(D, M, dtype)
    assert x[0].numel() > 2 ** 31 or x[2].numel() > 2 ** 31
    out, s, ckpt = cp.causal_product_fwd_delta(*x, return_state=True, save=True)
    grads = cp.causal_product_bwd_delta(*x, go, ckpt)
    del ckpt
    # rows of the end, from a state that the rows before it made (all but forgotten)
    lo = N - 2 * END
    y = [t[:, :, lo:].contiguous() for t in x]
    e_out, e_s, ckpt = cp.causal_product_fwd_delta(*y, return_state=True, save=True)
    e_grads = cp.causal_product_bwd_delta(*y, go[:, :, lo:].contiguous(), ckpt)
    for got, want in zip((out, *grads), (e_out, *e_grads)):
        a, b = got[:, :, N - END:].double(), want[:, :, END:].double()
        assert (a - b).norm() <= 1e-4 * b.norm()
    assert (s - e_s).norm() <= 1e-6 * e_s.norm()
    # and of the beginning, whose gradients no later row reaches
    y = [t[:, :, :2 * END].contiguous() for t in x]
    b_out, ckpt = cp.causal_product_fwd_delta(*y, save=True)
    b_grads = cp.causal_product_bwd_delta(*y, go[:, :, :2 * END].contiguous(), ckpt)
    for got, want in zip((out, *grads), (b_out, *b_grads)):
        a, b = got[:, :, :END].double(), want[:, :, :END].double()
        assert (a - b).norm() <= 1e-4 * b.norm()


def test_norm():
    B, H, n, D, R = 1, 18, (1 << 20) + 7, 128, 64
    gen = torch.Generator(device=DEV).manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    proj = rnd(B, n, (H + 1) * D)
    x = proj[..., :H * D].view(B, n, H, D).transpose(1, 2)
    k = proj[..., H * D:].view(B, n, 1, D).transpose(1, 2)
    assert x.numel() > 2 ** 31
    w = rnd(D)
    angle = torch.rand((n, R // 2), generator=gen, device=DEV) * 6
    cos, sin = angle.cos(), angle.sin()
    y, yk = cp.causal_product_qk_rope(x, k, w, w, cos, sin)
    dx, dxk = cp.causal_product_qk_rope_bwd(x, k, w, w, y, yk, cos, sin)[:2]
    lo = n - 500
    part = (x[:, :, lo:], k[:, :, lo:], w, w)
    z, zk = cp.causal_product_qk_rope(*part, cos[lo:], sin[lo:])
    dz, dzk = cp.causal_product_qk_rope_bwd(*part, z, zk, cos[lo:], sin[lo:])[:2]
    for a, b in ((y, z), (yk, zk), (dx, dz), (dxk, dzk)):
        assert torch.equal(a[:, :, lo:], b)
