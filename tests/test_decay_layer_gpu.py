"""Linear attention with a decay and the layer norm as a layer uses them
(``-m gpu``): norm of the rows, projections, the q/k norm with rotation, attention
with a decay per head, norm per head into token-major rows, projection, residual.

Training: the loss's gradients against the same layer in 64 bits.  Serving: a
padded batch of prompts into slots of a pool of states, then token by token,
against the layer over the whole sequences."""
import numpy as np
import pytest
import torch

import prefix_sum_outer_gb300 as cp
from test_decay_gpu import DEV

pytestmark = pytest.mark.gpu

H, HK, D, M, W = 4, 2, 64, 64, 256
G = -torch.exp2(-torch.arange(5, 5 + H, dtype=torch.float32))
SCALE = D ** -0.5


def weights(dtype, seed=1):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    p = {"n_w": 1 + 0.1 * rnd(W), "n_b": 0.1 * rnd(W), "qkv": rnd(W, (2 * HK * D + H * M)) / 16,
         "h_w": 1 + 0.1 * rnd(H, M), "h_b": 0.1 * rnd(H, M), "out": rnd(H * M, W) / 16}
    return {n: t.to(DEV, dtype) for n, t in p.items()}


def tables(N, dtype=torch.float32):
    ang = torch.arange(N, device=DEV, dtype=torch.float64)[:, None] * torch.exp(
        -torch.arange(8, device=DEV, dtype=torch.float64))
    return ang.cos().to(dtype), ang.sin().to(dtype)


def heads(x, p):
    B, N = x.shape[:2]
    y = cp.layer_norm(x, p["n_w"], p["n_b"]) @ p["qkv"]
    cut = lambda lo, n, d: y[..., lo:lo + n * d].view(B, N, n, d).transpose(1, 2)  # noqa: E731
    return cut(0, HK, D), cut(HK * D, HK, D), cut(2 * HK * D, H, M)


def layer(x, p, cos, sin, g=None, **kw):
    xq, xk, v = heads(x, p)
    q, k = cp.qk_rope(xq, xk, None, None, cos, sin, "l2")
    got = cp.causal_product_decay(q, k, v.contiguous(), G.to(DEV) if g is None else g, scale=SCALE, **kw)
    out, s = got if kw.get("return_state") else (got, None)
    y = cp.layer_norm(out, p["h_w"], p["h_b"], token_major=True).flatten(2)
    return x + y @ p["out"], s


def layer64(x, p, cos, sin):
    """The same in 64 bits, of torch's elementary operations."""
    def norm(t, w, b):
        d = t - t.mean(-1, keepdim=True)
        return d / (d.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w + b

    B, N = x.shape[:2]
    y = norm(x, p["n_w"], p["n_b"]) @ p["qkv"]
    cut = lambda lo, n, d: y[..., lo:lo + n * d].view(B, N, n, d).transpose(1, 2)  # noqa: E731

    def turn(t):
        t = t / (t.square().sum(-1, keepdim=True) + 1e-6).sqrt()
        h = cos.shape[-1]
        a, b, rest = t[..., :h], t[..., h:2 * h], t[..., 2 * h:]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, rest), -1).repeat_interleave(H // HK, 1)

    q, k, v = turn(cut(0, HK, D)), turn(cut(HK * D, HK, D)), cut(2 * HK * D, H, M)
    r = torch.arange(N, device=DEV)
    gap = (r[:, None] - r).double()
    w = torch.where(gap >= 0, torch.exp(G.to(DEV).double()[:, None, None] * gap.clamp_min(0)), 0.0)
    out = SCALE * ((q @ k.mT) * w) @ v
    y = norm(out, p["h_w"][:, None], p["h_b"][:, None]).transpose(1, 2).flatten(2)
    return x + y @ p["out"]


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-4), (torch.bfloat16, 4e-2)], ids=str)
def test_training(dtype, tol):
    """Gradients of every weight and of the input.  Bounds: in bf16 a rounding of
    2^-8 to each of the ten tensors on the way there and as many back; in fp32 the
    matrix products' own (tf32 is off), 1e-4 with room."""
    N = 300
    p = weights(dtype)
    gen = torch.Generator().manual_seed(2)
    x = torch.randn((2, N, W), generator=gen).to(DEV, dtype)
    t = torch.randn((2, N, W), generator=gen).to(DEV, dtype)
    leaves = {n: w.clone().requires_grad_(True) for n, w in (*p.items(), ("x", x))}
    cos, sin = tables(N)
    y, _ = layer(leaves["x"], leaves, cos, sin)
    y.backward(t)
    exact = {n: w.double().requires_grad_(True) for n, w in (*p.items(), ("x", x))}
    z = layer64(exact["x"], exact, *tables(N, torch.float64))
    z.backward(t.double())
    assert (y.double() - z).norm() <= tol * z.norm()
    for n in leaves:
        a, b = leaves[n].grad.double(), exact[n].grad
        assert (a - b).norm() <= tol * b.norm(), f"{n}: {float((a - b).norm() / b.norm()):.3g}"


@torch.no_grad()
def test_serving():
    """Prompts of 1 to 200 rows and 30 answered tokens each, bf16, against one
    padded run over all of it: the same arithmetic but for the chunks' rounding of
    bf16 results, 2^-8 a tensor."""
    dtype, lens, more = torch.bfloat16, [200, 1, 77, 128], 30
    B, N = len(lens), max(lens)
    p = weights(dtype)
    gen = torch.Generator().manual_seed(3)
    x = torch.randn((B, N + more, W), generator=gen).to(DEV, dtype)
    cos, sin = tables(N + more)
    whole, _ = layer(x, p, cos, sin)

    prompt = x[:, :N].clone()
    for b, n in enumerate(lens):
        prompt[b, n:] = float("nan")            # padding, whatever is in it
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    got, s = layer(prompt, p, cos[:N], sin[:N], return_state=True, lengths=n)
    for b, e in enumerate(lens):
        assert (got[b, :e] - whole[b, :e]).norm() <= 2e-2 * whole[b, :e].norm()
    pool = torch.zeros((7, H, D, M), device=DEV)
    slots = torch.tensor([5, 0, 3, 6], dtype=torch.int32, device=DEV)
    pool[slots.long()] = s
    at = n.long()
    for _ in range(more):
        row = x[torch.arange(B, device=DEV), at][:, None]
        xq, xk, v = heads(row, p)
        q, k = cp.qk_rope(xq, xk, None, None, cos[at][:, None], sin[at][:, None], "l2")
        o = cp.causal_product_decode_decay(q[:, :, 0], k[:, :, 0], v[:, :, 0].contiguous(), G.to(DEV), pool,
                                           scale=SCALE, slots=slots)
        y = cp.layer_norm(o[:, :, None], p["h_w"], p["h_b"], token_major=True).flatten(2)
        step = row + y @ p["out"]
        want = whole[torch.arange(B, device=DEV), at][:, None]
        assert (step - want).norm() <= 2e-2 * want.norm()
        at = at + 1
    assert not pool[[1, 2, 4]].any() and np.isfinite(float(pool.sum()))


def test_training_step_in_a_graph():
    """A whole step (forward, gradients by autograd) captured after a few on a side
    stream, replayed on new inputs: bitwise what the same step gives outside."""
    p = {n: t.requires_grad_() for n, t in weights(torch.bfloat16, seed=3).items()}
    cos, sin = tables(300)
    g = G.to(DEV)
    gen = torch.Generator(device=DEV).manual_seed(4)
    x, go = (torch.randn((2, 300, W), device=DEV, generator=gen).bfloat16() for _ in range(2))

    def step():
        for t in p.values():
            t.grad = None
        y, _ = layer(x, p, cos, sin, g)
        y.backward(go)
        return y.detach(), [t.grad for t in p.values()]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, grads = step()
    for t in (x, go):
        t.copy_(torch.randn(t.shape, device=DEV, generator=gen))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (y, *grads)]
    want, grads = step()
    for a, b in zip(got, (want, *grads)):
        assert torch.equal(a, b)
