"""The layer norm on the GPU (``-m gpu``) against its 64-bit reference.

Bounds: y and dx element by element, one rounding to the output's type (half a
step: bf16 2^-8 of the value's binade, fp16 2^-11, fp32 2^-24) and fp32 arithmetic
before it: sums of C terms in registers and shuffles (fewer than 16 + log2 C
roundings of 2^-24 of a partial sum, 2e-6 of what is summed in absolute value)
and a few roundings of each term.  dw and db are sums over rows, in fp32: 2^-24 of
the sum of absolute values a rounding, of which a sum of R rows has at most
about R / 64 + 200 in line (a group of threads sums its rows one after the
other), so 2e-6 of that sum where R is a few thousand."""
import numpy as np
import pytest
import torch

import decay_reference as ref
import prefix_sum_outer_gb300 as cp

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(lead, C, dt, seed, per_head=False, weights=True):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    wide = (lead[1], C) if per_head else (C,)
    x = {"x": (1.5 * rnd(*lead, C) + rnd(*lead, 1)).to(DT[dt]),
         "w": (1 + 0.3 * rnd(*wide)).to(DT[dt]) if weights else None,
         "b": (0.3 * rnd(*wide)).to(DT[dt]) if weights else None, "gy": rnd(*lead, C).to(DT[dt])}
    return {n: None if t is None else t.to(DEV) for n, t in x.items()}


def near(got, want, scale, name):
    """|got - want| <= half a step of the type + 2e-6 of ``scale``."""
    got = got.detach()
    want_t = torch.from_numpy(np.ascontiguousarray(want))
    assert got.shape == want_t.shape, name
    step = torch.finfo(got.dtype).eps / 2
    bound = step * want_t.abs().clamp_min(torch.finfo(got.dtype).tiny) + 2e-6 * torch.as_tensor(scale)
    off = (got.double().cpu() - want_t).abs()
    assert bool((off <= bound).all()), f"{name}: {float((off / bound).max()):.3g} of the bound"


def check(x, major=False, per_head=False):
    kw = dict(eps=EPS, token_major=major)
    gy = x["gy"].transpose(1, 2).contiguous() if major else x["gy"]
    y = cp.causal_product_layer_norm(x["x"], x["w"], x["b"], **kw)
    dx, dw, db = cp.causal_product_layer_norm_bwd(x["x"], x["w"], x["b"], gy, **kw)
    torch.cuda.synchronize()
    turn = lambda t: t.transpose(1, 2) if major else t  # noqa: E731
    a = f64(x["x"])
    wide = lambda t: None if t is None else (f64(t)[:, None] if per_head else f64(t))  # noqa: E731
    w, b = wide(x["w"]), wide(x["b"])
    # rows' own sizes: values of xh are ~1, and mu may be large beside the spread
    spread = np.sqrt(a.var(-1, keepdims=True) + EPS)
    lift = 1.0 + np.abs(a).max(-1, keepdims=True) / spread
    r_y = ref.layer_norm_fwd(a, w, b, EPS)
    near(turn(y), r_y, lift * (1.0 + np.abs(r_y)), "y")
    g = f64(x["gy"])
    r_dx, t_w, t_b = ref.layer_norm_bwd(a, w, EPS, g)
    big = np.abs(g).max(-1, keepdims=True) * (1.0 if w is None else np.abs(w).max())
    near(dx, r_dx, lift * big * (2.0 + np.abs(r_dx * spread)) / spread, "dx")
    assert y.is_contiguous() and dx.is_contiguous()
    over = (0, 2) if per_head else tuple(range(a.ndim - 1))
    # a term gy xh is off by |gy| times what xh is off by, which is y's bound: the
    # error of mu, 2^-24 of the row's values, stays where xh = (x - mu) r is near 0
    for got, t, scale in ((dw, t_w, np.abs(g) * lift + np.abs(t_w) * lift), (db, t_b, np.abs(t_b))):
        if x["w"] is None:
            assert got is None
        else:
            near(got, t.sum(over), scale.sum(over), "dw or db")
    return y, dx, dw, db


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,C", [
    (1, 1), (3, 2), (5, 7), (1, 8), (2, 16), (33, 24), (17, 31), (40, 32), (9, 40), (65, 64), (21, 65),
    (30, 96), (7, 128), (12, 130), (50, 200), (11, 256), (6, 257), (19, 500), (8, 512), (5, 513),
    (700, 1000), (40, 1024), (3, 1030), (10, 2048), (4, 2051), (6, 4096), (3, 5000), (2, 8192),
    (3, 8200), (2, 12149), (2, 16384), (1, 16385), (2, 20000), (1, 32768), (2, 32767)],
    ids=lambda v: str(v))
def test_rows(rows, C, dt):
    check(make((rows,), C, dt, seed=rows + C))


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("B,H,N,C", [(1, 1, 1, 64), (61, 16, 1, 64), (2, 3, 37, 64), (3, 5, 50, 40),
                                     (2, 4, 33, 128), (1, 2, 9, 72), (2, 3, 8, 33), (1, 3, 20, 1024),
                                     (2, 2, 5, 2056)])
def test_heads(B, H, N, C, per_head, dt):
    x = make((B, H, N), C, dt, seed=B + H + N + C, per_head=per_head)
    a = check(x, major=True, per_head=per_head)
    b = check(x, major=False, per_head=per_head)
    assert torch.equal(a[0].transpose(1, 2), b[0])
    for s, t in zip(a[1:], b[1:]):
        assert torch.equal(s, t)


def test_many_rows():
    """More rows than the card holds at a time, whose sums go through many parts."""
    check(make((2, 40000), 64, "f32", seed=1))
    check(make((4, 3, 9000), 64, "bf16", seed=2, per_head=True), major=True, per_head=True)
    check(make((5000,), 1024, "bf16", seed=3))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_with_parts_of_the_arguments(dt):
    x = make((3, 20), 96, dt, seed=4, weights=False)
    check(x)
    full = make((3, 20), 96, dt, seed=5)
    kw = dict(eps=EPS)
    y = cp.causal_product_layer_norm(full["x"], full["w"], **kw)
    z = cp.causal_product_layer_norm(full["x"], full["w"], torch.zeros_like(full["w"]), **kw)
    assert torch.equal(y, z)
    dx, dw, db = cp.causal_product_layer_norm_bwd(full["x"], full["w"], None, full["gy"], **kw)
    ex, ew, eb = cp.causal_product_layer_norm_bwd(full["x"], full["w"], full["b"], full["gy"], **kw)
    assert torch.equal(dx, ex) and torch.equal(dw, ew) and db is None
    ones = torch.ones_like(full["w"])
    dx, dw, db = cp.causal_product_layer_norm_bwd(full["x"], None, full["b"], full["gy"], **kw)
    ex, _, fb = cp.causal_product_layer_norm_bwd(full["x"], ones, full["b"], full["gy"], **kw)
    assert torch.equal(dx, ex) and dw is None and torch.equal(db, fb) and torch.equal(db, eb)


@pytest.mark.parametrize("C", [64, 1024, 4096])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_layouts(dt, C):
    """Token-major rows seen head-major, rows at odd strides and addresses
    (element loads) and a broadcast batch give the dense rows' numbers."""
    x = make((2, 3, 23), C, dt, seed=6)
    want = cp.causal_product_layer_norm(x["x"], x["w"], x["b"])
    d_want = cp.causal_product_layer_norm_bwd(x["x"], x["w"], x["b"], x["gy"])
    major = x["x"].transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(cp.causal_product_layer_norm(major, x["w"], x["b"]), want)
    for a, b in zip(cp.causal_product_layer_norm_bwd(major, x["w"], x["b"], x["gy"]), d_want):
        assert torch.equal(a, b)
    buf = torch.zeros(2, 3, 23, C + 3, dtype=x["x"].dtype, device=DEV)
    buf[..., 1:C + 1] = x["x"]
    check(dict(x, x=buf[..., 1:C + 1]))
    odd = torch.zeros(C + 1, dtype=x["x"].dtype, device=DEV)
    odd[1:] = x["w"]
    check(dict(x, w=odd[1:]))
    one = x["x"][:1].expand(2, -1, -1, -1)
    y = cp.causal_product_layer_norm(one, x["w"], x["b"])
    assert torch.equal(y[0], want[0]) and torch.equal(y[1], want[0])


def test_extremes():
    """A constant row gives the bias; a row with a large mean keeps its
    variance; inf and NaN stay in their row, and reach the weights' gradients."""
    x = make((12,), 64, "f32", seed=7)
    x["x"][0] = 3.0
    x["x"][1] = 1000.0 + 0.5 * x["x"][1]
    x["x"][2] *= 1e-18
    x["x"][3] *= 1e15
    y, dx, _, _ = check(x)
    assert torch.equal(y[0], x["b"])
    x["x"][5, 3], x["x"][7, 60] = float("inf"), float("nan")
    z = cp.causal_product_layer_norm(x["x"], x["w"], x["b"], EPS)
    dz, dw, db = cp.causal_product_layer_norm_bwd(x["x"], x["w"], x["b"], x["gy"], EPS)
    rest = [i for i in range(12) if i not in (5, 7)]
    assert torch.equal(z[rest], y[rest]) and torch.equal(dz[rest], dx[rest])
    assert torch.isnan(z[5]).any() and torch.isnan(z[7]).all() and torch.isnan(dz[7]).all()
    assert torch.isnan(dw).any() and torch.isfinite(db).all()


def test_no_rows():
    w = torch.ones(16, device=DEV)
    for shape in ((0, 16), (2, 0, 16), (2, 3, 0, 16)):
        e = torch.empty(shape, device=DEV)
        assert cp.causal_product_layer_norm(e, w, w).shape == shape
        dx, dw, db = cp.causal_product_layer_norm_bwd(e, w, w, e)
        assert dx.shape == shape and not dw.any() and not db.any()


def test_autograd_against_differences():
    """Directional central differences of the fp32 forward (h = 1e-2: h^2 of the
    third derivative, of size 1, and 1e-6 of the result over h)."""
    x = make((2, 3, 9), 32, "f32", seed=8, per_head=True)
    leaves = [x[n].clone().requires_grad_(True) for n in ("x", "w", "b")]
    gy = x["gy"].transpose(1, 2).contiguous()

    def loss(a):
        return (cp.layer_norm(*a, EPS, True).double() * gy.double()).sum()

    grads = torch.autograd.grad(loss(leaves), leaves)
    gen = torch.Generator(device=DEV).manual_seed(1)
    for i, g in enumerate(grads):
        way = torch.randn(g.shape, generator=gen, device=DEV)
        way = way / way.norm()
        with torch.no_grad():
            up, down = (loss([t + s * 1e-2 * way if j == i else t for j, t in enumerate(leaves)])
                        for s in (1, -1))
        assert abs((up - down) / 2e-2 - (g.double() * way).sum()) <= 2e-3 * g.double().norm()
    # a gradient that is not dense, an input that needs none
    y = cp.layer_norm(x["x"], leaves[1], None)
    (dw,) = torch.autograd.grad(y, leaves[1], x["gy"].transpose(2, 3).contiguous().transpose(2, 3))
    assert torch.equal(dw, cp.causal_product_layer_norm_bwd(x["x"], x["w"], None, x["gy"])[1])


@pytest.mark.parametrize("dt,C", [("bf16", 64), ("f32", 1000), ("f16", 4096)])
def test_repeatable_streams_buffers_and_graphs(dt, C):
    x = make((3, 4, 70), C, dt, seed=9)
    gy = x["gy"].transpose(1, 2).contiguous()
    pad = 1024
    n = x["x"].numel()
    buf = torch.full((n + 2 * pad,), 7.0, dtype=DT[dt], device=DEV)
    out = buf[pad:pad + n].view(3, 70, 4, C)
    size = cp.load_library().causal_product_layer_norm_workspace_size(3, 4, 70, C, cp._DTYPES[DT[dt]])
    space = torch.full((size + 256,), 7, dtype=torch.uint8, device=DEV)

    def run(stream=None):
        return [cp.causal_product_layer_norm(x["x"], x["w"], x["b"], token_major=True, out=out, stream=stream),
                *cp.causal_product_layer_norm_bwd(x["x"], x["w"], x["b"], gy, token_major=True,
                                                  workspace=space[:size], stream=stream)]

    first = [t.clone() for t in run()]
    torch.cuda.synchronize()
    assert (buf[:pad] == 7).all() and (buf[-pad:] == 7).all() and (space[size:] == 7).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = run(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = run()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_refusals():
    x = make((2, 3, 5), 64, "bf16", seed=10)
    f = cp.causal_product_layer_norm
    with pytest.raises(ValueError):
        f(x["x"][0], token_major=True)
    with pytest.raises(ValueError):
        f(x["x"].reshape(-1))
    with pytest.raises(ValueError):
        f(x["x"], x["w"][:32])
    with pytest.raises(ValueError):
        f(x["x"], torch.ones(5, 64, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        f(x["x"], torch.ones(3, 64, dtype=torch.bfloat16, device=DEV), x["b"])   # two shapes
    with pytest.raises(ValueError):
        f(x["x"].transpose(2, 3))                                                # rows not dense
    with pytest.raises(TypeError):
        f(x["x"], x["w"].float())
    with pytest.raises(TypeError):
        f(x["x"].double())
    with pytest.raises(RuntimeError):
        f(x["x"], x["w"].cpu())
    with pytest.raises(ValueError):
        f(x["x"], out=torch.empty(2, 3, 5, 64, device=DEV))
    with pytest.raises(cp.CausalProductError):
        f(x["x"], out=x["x"])
    with pytest.raises(cp.CausalProductError):
        f(x["x"], eps=-1.0)
    with pytest.raises(cp.CausalProductError):
        f(torch.zeros(2, 32769, device=DEV))
    with pytest.raises(ValueError):
        cp.causal_product_layer_norm_bwd(x["x"], x["w"], x["b"], x["gy"][:1])
    with pytest.raises(ValueError):
        cp.causal_product_layer_norm_bwd(x["x"], x["w"], x["b"], x["gy"], token_major=True)
    with pytest.raises(ValueError):
        cp.causal_product_layer_norm_bwd(x["x"], x["w"], x["b"], x["gy"].transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(cp.CausalProductError):
        cp.causal_product_layer_norm_bwd(x["x"], x["w"], x["b"], x["gy"],
                                         workspace=torch.zeros(256, dtype=torch.uint8, device=DEV))
