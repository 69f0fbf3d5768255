"""Tensors that are dense but start off a 16-byte boundary, through the autograd
wrappers (``-m gpu``): the gradient of a torch.cat or torch.stack of odd-sized
results is such a view, as a slice of a batch is.  The C entry points want whole
16-byte addresses; the wrappers copy what has none, and the results are the bits
that the same values give at an aligned address."""
import pytest
import torch

import prefix_sum_outer_gb300 as cp
from test_decay_gpu import DEV, DT

pytestmark = pytest.mark.gpu


def rnd(shape, dt, seed, grad=False):
    gen = torch.Generator().manual_seed(seed)
    t = torch.randn(shape, generator=gen).to(dt).to(DEV)
    return t.requires_grad_(True) if grad else t


def off(t):
    """The same values one element off a boundary."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    flat[1:] = t.detach().reshape(-1)
    got = flat[1:].view(t.shape)
    assert got.is_contiguous() and got.data_ptr() % 16
    return got.requires_grad_(t.requires_grad)


@pytest.mark.parametrize("dt,C", [("f32", 5), ("bf16", 33), ("f16", 7), ("bf16", 64)])
def test_layer_norm_of_joined_rows(dt, C):
    a, b = rnd((3, C), DT[dt], 1, True), rnd((4, C), DT[dt], 2, True)
    w, bias = rnd((C,), DT[dt], 3, True), rnd((C,), DT[dt], 4, True)
    gy = rnd((7, C), DT[dt], 5)
    joined = torch.cat([cp.layer_norm(a, w, bias), cp.layer_norm(b, w, bias)])
    da, db = torch.autograd.grad(joined, (a, b), gy, retain_graph=True)
    for x, lo, hi, d in ((a, 0, 3, da), (b, 3, 7, db)):
        want = torch.autograd.grad(cp.layer_norm(x, w, bias), x, gy[lo:hi].clone())[0]
        assert torch.equal(d, want)
    dw = torch.autograd.grad(joined, w, gy)[0]
    parts = [torch.autograd.grad(cp.layer_norm(x, w, bias), w, g.clone())[0]
             for x, g in ((a, gy[:3]), (b, gy[3:]))]
    assert torch.allclose(dw, parts[0] + parts[1])


def both(call, inputs, grads, inputs_too=True):
    """The call's results and gradients from the tensors as they are and from
    unaligned copies of them, with gradients to match."""
    got = []
    fresh = lambda t: t.detach().clone().requires_grad_(t.requires_grad)  # noqa: E731
    for place in (fresh, off):
        x = [(place if inputs_too else fresh)(t) for t in inputs]
        outs = call(*x)
        outs = outs if isinstance(outs, tuple) else (outs,)
        leaves = [t for t in x if t.requires_grad]
        d = torch.autograd.grad(outs, leaves, [place(g) for g in grads])
        with torch.no_grad():
            plain = call(*x)
        plain = plain if isinstance(plain, tuple) else (plain,)
        got.append((*outs, *d, *plain))
    assert len(got[0]) == len(got[1])
    for i, (a, b) in enumerate(zip(*got)):
        assert torch.equal(a, b), i


@pytest.mark.parametrize("dt,D,M", [("f32", 33, 5), ("f16", 65, 33), ("bf16", 64, 64)])
def test_decay(dt, D, M):
    B, H, Hk, N, t = 2, 4, 2, 70, DT[dt]
    g = -torch.rand(H, generator=torch.Generator().manual_seed(9)).to(DEV)
    n = torch.tensor([70, 41], dtype=torch.int32, device=DEV)
    both(lambda q, k, v, s: cp.causal_product_decay(q, k, v, g, state=s, return_state=True,
                                                    scale=0.3, lengths=n),
         [rnd((B, Hk, N, D), t, 1, True), rnd((B, Hk, N, D), t, 2, True),
          rnd((B, H, N, M), t, 3, True), rnd((B, H, D, M), torch.float32, 4, True)],
         [rnd((B, H, N, M), t, 5), rnd((B, H, D, M), torch.float32, 6)])


def test_decay_of_a_slice_of_the_batch():
    """q[1:], state[1:] of odd widths: dense views."""
    q, k, v = (rnd((3, 2, 5, 33), torch.float32, i) for i in (1, 2, 3))
    s, g = rnd((3, 2, 33, 33), torch.float32, 4), torch.full((2,), -0.1, device=DEV)
    got = cp.causal_product_decay(q[1:], k[1:], v[1:], g, state=s[1:], return_state=True)
    want = cp.causal_product_decay(q, k, v, g, state=s, return_state=True)
    for a, b in zip(got, want):
        assert torch.equal(a, b[1:])


@pytest.mark.parametrize("dt,D,M", [("f32", 33, 5), ("f16", 65, 33)])
def test_the_other_products(dt, D, M):
    B, H, N, t = 2, 2, 70, DT[dt]
    q, k, v = rnd((B, H, N, D), t, 1, True), rnd((B, H, N, D), t, 2, True), rnd((B, H, N, M), t, 3, True)
    s, go, gs = rnd((B, H, D, M), torch.float32, 4, True), rnd((B, H, N, M), t, 5), \
        rnd((B, H, D, M), torch.float32, 6)
    both(cp.causal_product, [q, k, v], [go])
    both(lambda q, k, v: cp.causal_product(q, k, v, feature="elu1"), [q, k, v], [go])
    both(lambda q, k, v, s: cp.causal_product(q, k, v, state=s, return_state=True), [q, k, v, s],
         [go, gs])
    g, beta = -rnd((B, H, N), torch.float32, 8).abs().detach(), rnd((B, H, N), torch.float32, 9).sigmoid()
    unit = k.detach() / k.detach().float().norm(dim=-1, keepdim=True).to(t)
    both(lambda q, k, v, g, b, s: cp.causal_product_delta(q, k, v, g, b, state=s, return_state=True),
         [q, unit.requires_grad_(True), v, g.requires_grad_(True), beta.detach().requires_grad_(True), s],
         [go, gs])


@pytest.mark.parametrize("dt,D", [("f32", 33), ("f16", 64)])  # (16-bit: multiples of 8)
def test_normalizer(dt, D):
    both(cp.normalizer, [rnd((2, 2, 71, D), DT[dt], 1, True), rnd((2, 2, 71, D), DT[dt], 2, True)],
         [rnd((2, 2, 71), torch.float32, 3)])


def test_qk_rope():
    xq, xk = rnd((2, 3, 5, 40), torch.float32, 1, True), rnd((2, 1, 5, 40), torch.float32, 2, True)
    both(lambda a, b: cp.qk_rope(a, b), [xq, xk],
         [rnd((2, 3, 5, 40), torch.float32, 3), rnd((2, 1, 5, 40), torch.float32, 4)],
         inputs_too=False)  # (rows of any alignment are read in place)
