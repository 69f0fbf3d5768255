"""The q/k norm with rotation on the GPU (``-m gpu``) against its 64-bit
reference.  Bounds as for the other operators: one rounding to the output's
type (bf16 2^-8, fp16 2^-11) and at most 1e-5 of fp32 arithmetic before it
(sums of up to 256 squares; a weight's gradient sums up to a few thousand
rows)."""
import numpy as np
import pytest
import torch

import delta_reference as ref
import prefix_sum_outer_gb300 as cp
from test_delta_gpu import DEV, DT, close, f64

pytestmark = pytest.mark.gpu


def make(B, Hq, Hk, N, D, R, dt, seed, weights=True, shared=False):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    proj = (rnd(B, N, (Hq + 2 * Hk) * D) * 2).to(DT[dt]).to(DEV)
    x = {"xq": proj[..., :Hq * D].view(B, N, Hq, D).transpose(1, 2),
         "xk": proj[..., Hq * D:(Hq + Hk) * D].view(B, N, Hk, D).transpose(1, 2)}
    for n, H in (("wq", Hq), ("wk", Hk)):
        x[n] = (1 + 0.3 * rnd(D)).to(DT[dt]).to(DEV) if weights else None
        x["g" + n[1]] = rnd(B, H, N, D).to(DT[dt]).to(DEV)
    ang = 3 * rnd(*((N, R // 2) if shared else (B, N, R // 2))).to(DEV)
    x["cos"], x["sin"] = torch.cos(ang), torch.sin(ang)
    return x


def check(x, norm, eps=1e-5):
    kw = dict(norm=norm, eps=eps)
    a = (x["xq"], x["xk"], x["wq"], x["wk"])
    q, k = cp.causal_product_qk_rope(*a, x["cos"], x["sin"], **kw)
    dxq, dxk, dwq, dwk = cp.causal_product_qk_rope_bwd(*a, x["gq"], x["gk"], x["cos"], x["sin"], **kw)
    torch.cuda.synchronize()
    B, _, N, _ = x["xq"].shape
    cos, sin = (np.broadcast_to(f64(t), (B, N, t.shape[-1])) for t in (x["cos"], x["sin"]))
    for xx, w, gy, y, dx, dw in ((x["xq"], x["wq"], x["gq"], q, dxq, dwq),
                                 (x["xk"], x["wk"], x["gk"], k, dxk, dwk)):
        r_dx, r_dw = ref.qk_rope_bwd(f64(xx), f64(w), cos, sin, norm, eps, f64(gy))
        close(y, ref.qk_rope_fwd(f64(xx), f64(w), cos, sin, norm, eps), "y")
        close(dx, r_dx, "dx")
        assert y.is_contiguous() and dx.is_contiguous()
        if w is None:
            assert dw is None
        else:
            close(dw, r_dw, "dw")


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("shape", [
    (1, 1, 1, 1, 8, 0, "bf16"), (61, 4, 2, 1, 64, 64, "f16"), (2, 3, 1, 37, 64, 16, "bf16"),
    (1, 2, 2, 50, 128, 128, "bf16"), (2, 2, 1, 19, 96, 32, "bf16"), (1, 2, 2, 33, 40, 40, "f16"),
    (1, 2, 1, 21, 72, 14, "f32"), (2, 1, 1, 30, 256, 64, "f32"), (1, 5, 3, 17, 24, 2, "bf16"),
    (1, 16, 4, 700, 64, 64, "bf16"), (1, 2, 2, 9, 248, 130, "f16")],
    ids=lambda s: "x".join(map(str, s)))
def test_against_reference(shape, norm):
    *dims, dt = shape
    check(make(*dims, dt, seed=sum(dims)), norm)


def test_without_weights_and_with_one_table():
    check(make(3, 2, 2, 20, 64, 32, "bf16", 1, weights=False, shared=True), "l2")
    x = make(2, 2, 2, 20, 64, 32, "f32", 2, shared=True)
    x["wk"] = None
    check(x, "rms")


def test_layouts():
    """Dense rows, rows at odd strides (element loads) and a broadcast batch
    give the bits of the strided view."""
    x = make(2, 2, 1, 23, 64, 16, "bf16", 3)
    kw = dict(cos=x["cos"], sin=x["sin"])
    want = cp.causal_product_qk_rope(x["xq"], x["xk"], x["wq"], x["wk"], **kw)
    dense = cp.causal_product_qk_rope(x["xq"].contiguous(), x["xk"].contiguous(), x["wq"], x["wk"], **kw)
    odd = []
    for t in (x["xq"], x["xk"]):
        B, H, N, D = t.shape
        buf = torch.zeros(B, H, N, D + 3, dtype=t.dtype, device=DEV)
        buf[..., 1:D + 1] = t
        odd.append(buf[..., 1:D + 1])
    at_odd = cp.causal_product_qk_rope(*odd, x["wq"], x["wk"], **kw)
    for a, b, c in zip(want, dense, at_odd):
        assert torch.equal(a, b) and torch.equal(a, c)
    one = cp.causal_product_qk_rope(x["xq"][:1].expand(2, -1, -1, -1), x["xk"][:1].expand(2, -1, -1, -1),
                                    x["wq"], x["wk"], x["cos"][0], x["sin"][0])
    assert torch.equal(one[0][0], one[0][1])


def test_zero_rows_and_extremes():
    """A zero row gives zeros and finite gradients; rows of large and small
    values keep their norm; inf and NaN stay in their row."""
    x = make(1, 2, 1, 12, 64, 64, "f32", 4)
    xq = x["xq"].contiguous()
    xq[0, 0, 0] = 0
    xq[0, 0, 1] *= 1e15
    xq[0, 0, 2] *= 1e-12
    xq[0, 1, 3, 5] = float("inf")
    a = (xq, x["xk"], x["wq"], x["wk"])
    q, _ = cp.causal_product_qk_rope(*a, x["cos"], x["sin"])
    dq = cp.causal_product_qk_rope_bwd(*a, x["gq"], x["gk"], x["cos"], x["sin"])[0]
    assert not q[0, 0, 0].any() and torch.isfinite(dq[0, 0]).all()
    bad = torch.zeros(12, dtype=torch.bool, device=DEV)
    bad[3] = True
    assert torch.equal(~torch.isfinite(q[0, 1]).all(-1), bad)
    assert torch.isfinite(dq[0, 1][~bad]).all()
    cos, sin = f64(x["cos"]), f64(x["sin"])
    for n in (1, 2):
        close(q[:, :1, n:n + 1], ref.qk_rope_fwd(f64(xq[:, :1, n:n + 1]), f64(x["wq"]), cos[:, n:n + 1],
                                                 sin[:, n:n + 1], "rms", 1e-6))


def test_autograd_against_differences():
    """Directional central differences of the fp32 forward (h = 1e-2)."""
    x = make(2, 2, 1, 9, 32, 16, "f32", 5)
    leaves = [x[n].clone().requires_grad_(True) for n in ("xq", "xk", "wq", "wk")]

    def loss(a):
        q, k = cp.qk_rope(*a, x["cos"], x["sin"], "rms", 1e-3)
        return (q.double() * x["gq"].double()).sum() + (k.double() * x["gk"].double()).sum()

    grads = torch.autograd.grad(loss(leaves), leaves)
    gen = torch.Generator(device=DEV).manual_seed(1)
    for i, g in enumerate(grads):
        way = torch.randn(g.shape, generator=gen, device=DEV)
        way = way / way.norm()
        with torch.no_grad():
            up, down = (loss([t + s * 1e-2 * way if j == i else t for j, t in enumerate(leaves)])
                        for s in (1, -1))
        assert abs((up - down) / 2e-2 - (g.double() * way).sum()) <= 2e-3 * g.double().norm()


def test_no_rows():
    e = torch.empty(2, 2, 0, 16, device=DEV)
    w = torch.ones(16, device=DEV)
    q, k = cp.causal_product_qk_rope(e, e, w, w)
    assert q.shape == e.shape
    d = cp.causal_product_qk_rope_bwd(e, e, w, w, e, e)
    assert not d[2].any() and not d[3].any()


def test_refusals():
    x = make(1, 2, 1, 6, 64, 16, "bf16", 6)
    f = cp.causal_product_qk_rope
    a = (x["xq"], x["xk"], x["wq"], x["wk"])
    with pytest.raises(ValueError):
        f(*a, x["cos"], None)
    with pytest.raises(ValueError):
        f(*a, x["cos"][:, :5], x["sin"][:, :5])
    with pytest.raises(ValueError):
        f(*a, x["cos"].half(), x["sin"].half())
    with pytest.raises(ValueError):
        f(*a, x["cos"], x["sin"], norm="max")
    with pytest.raises(ValueError):
        f(x["xq"], x["xk"][..., :32], x["wq"], x["wk"])
    with pytest.raises(ValueError):
        f(x["xq"], x["xk"], x["wq"][:32], x["wk"])
    with pytest.raises(TypeError):
        f(x["xq"], x["xk"], x["wq"].float(), x["wk"])
    with pytest.raises(ValueError):
        f(x["xq"].transpose(2, 3).contiguous().transpose(2, 3), x["xk"], x["wq"], x["wk"])
    with pytest.raises(RuntimeError):
        f(x["xq"], x["xk"], x["wq"].cpu(), x["wk"])
    with pytest.raises(cp.CausalProductError):
        f(*a, eps=-1.0)
    with pytest.raises(cp.CausalProductError):
        f(*a, torch.ones(6, 40, device=DEV), torch.ones(6, 40, device=DEV))  # R = 80 > 64
    with pytest.raises(cp.CausalProductError):
        f(x["xq"][..., :60], x["xk"][..., :60])
    dense = x["xq"].contiguous()
    with pytest.raises(cp.CausalProductError):
        f(dense, x["xk"], x["wq"], x["wk"], q=dense)
    with pytest.raises(ValueError):
        cp.causal_product_qk_rope_bwd(*a, x["gq"][:, :1], x["gk"])
