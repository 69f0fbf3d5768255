"""The gated delta rule on the GPU (``-m gpu``): the chunked forward and
backward and the one-token step against the 64-bit recurrence.

Errors are the 2-norm of the difference over the 2-norm of the result.  Bounds,
set by the arithmetic: a result rounded once to bf16 (8 significant bits) is at
most 2^-8 = 3.9e-3 off, to fp16 (11 bits) 2^-11 = 4.9e-4, and the computation
before that rounding adds at most 1e-5 where a factor is held as two bf16 numbers (16 bits, 2^-17 =
7.6e-6 each, of random sign) or in fp32 (sums of a few hundred products)."""
import numpy as np
import pytest
import torch

import delta_reference as ref
import prefix_sum_outer_gb300 as cp

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TOL = {torch.bfloat16: 2.0 ** -8 + 1e-5, torch.float16: 2.0 ** -11 + 1e-5, torch.float32: 1e-5}


def err(got, want):
    got = got.detach().double().cpu().numpy()
    assert got.shape == want.shape
    n = np.linalg.norm(want)
    d = np.linalg.norm(got - want)
    return d / n if n else d


def close(got, want, name=""):
    e = err(got, want)
    assert e <= TOL[got.dtype], f"{name}: {e:.3g} > {TOL[got.dtype]:.3g}"


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(B, H, Hk, N, D, M, dt, seed, carry=False, common=0.5, rate=0.3):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    q, k = unit(rnd(B, Hk, N, D)), unit(rnd(B, Hk, N, D) + common * rnd(1, Hk, 1, D))
    x = {"q": q.to(dt), "k": k.to(dt), "v": rnd(B, H, N, M).to(dt),
         "g": -rate * torch.rand((B, H, N), generator=gen), "beta": torch.rand((B, H, N), generator=gen),
         "go": rnd(B, H, N, M).to(dt), "s0": rnd(B, H, D, M) if carry else None,
         "gs": rnd(B, H, D, M) if carry else None}
    return {n: None if t is None else t.to(DEV) for n, t in x.items()}


def args(x):
    return [x[n] for n in ("q", "k", "v", "g", "beta")]


def check(x, scale=0.3):
    carry = x["s0"] is not None
    out, s, ckpt = cp.causal_product_fwd_delta(*args(x), state_in=x["s0"], return_state=True,
                                               scale=scale, save=True)
    d = cp.causal_product_bwd_delta(*args(x), x["go"], ckpt, scale=scale, grad_state_out=x["gs"],
                                    return_state_grad=True)
    plain = cp.causal_product_fwd_delta(*args(x), state_in=x["s0"], scale=scale)
    torch.cuda.synchronize()
    a = [f64(t) for t in args(x)]
    r_out, r_s, _ = ref.delta_fwd(*a, scale, f64(x["s0"]))
    r_d = ref.delta_bwd(*a, scale, f64(x["go"]), f64(x["gs"]), f64(x["s0"]))
    close(out, r_out, "out")
    close(s, r_s, "state")
    assert torch.equal(plain, out)
    for got, want, name in zip(d, r_d, ("dq", "dk", "dv", "dg", "dbeta", "dstate")):
        if name != "dstate" or carry:
            close(got, want, name)
    return out, s, d


# B, H, Hk, N, D, M, dtype, carried state
SHAPES = [
    (1, 1, 1, 1, 8, 8, "bf16", False), (2, 2, 1, 1, 64, 64, "bf16", True),
    (1, 2, 2, 63, 64, 64, "bf16", False), (1, 2, 2, 64, 64, 64, "bf16", True),
    (1, 2, 1, 65, 64, 64, "bf16", True), (1, 2, 2, 200, 64, 128, "bf16", False),
    (1, 2, 2, 150, 128, 64, "bf16", True), (1, 4, 1, 129, 128, 128, "bf16", True),
    (1, 2, 2, 97, 40, 72, "bf16", True), (1, 1, 1, 130, 96, 16, "bf16", True),
    (1, 1, 1, 70, 16, 200, "bf16", True), (1, 1, 1, 40, 256, 64, "bf16", True),
    (2, 2, 2, 33, 64, 64, "f32", True), (1, 4, 2, 70, 64, 128, "f32", True),
    (1, 1, 1, 37, 5, 3, "f32", True), (1, 1, 1, 40, 256, 40, "f32", True),
    (1, 3, 3, 65, 64, 64, "f16", True), (1, 2, 1, 40, 72, 24, "f16", False),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward_and_backward(shape):
    B, H, Hk, N, D, M, dt, carry = shape
    check(make(B, H, Hk, N, D, M, DT[dt], seed=N + D + M, carry=carry))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_correlated_keys_and_full_strength(dt):
    """Keys that all but coincide, written at full strength with no decay: the
    triangular system's entries are all near 1."""
    x = make(1, 2, 2, 190, 64, 64, DT[dt], seed=5, carry=True, common=4.0, rate=0.0)
    x["beta"].fill_(1.0)
    check(x)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_cleared_states_and_padding(dt):
    """-inf clears the state (also at the first token and twice in a chunk);
    g = beta = 0 is padding; a fully padded head keeps its state."""
    x = make(1, 3, 3, 140, 64, 64, DT[dt], seed=6, carry=True)
    x["g"][:, 0, [0, 20, 21, 70, 139]] = -np.inf
    x["g"][:, 1, 30:90], x["beta"][:, 1, 30:90] = 0.0, 0.0
    x["g"][:, 2], x["beta"][:, 2] = 0.0, 0.0
    out, s, d = check(x)
    assert torch.equal(s[:, 2], x["s0"][:, 2])
    assert torch.equal(d[3][:, 0, [0, 20, 21, 70, 139]], torch.zeros((1, 5), device=DEV))
    assert not d[2][:, 2].any() and not d[5][:, 0].any()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_large_decays(dt):
    """Decays between e^-60 and e^-100 at every token, whose running sums pass
    the exponent range of fp32."""
    x = make(1, 2, 2, 100, 64, 64, DT[dt], seed=7, carry=True)
    x["g"][:] = -60.0 - 40.0 * torch.rand(x["g"].shape, device=DEV)
    x["g"][:, 1, ::3] = -0.01
    out, s, ckpt = cp.causal_product_fwd_delta(*args(x), state_in=x["s0"], return_state=True, save=True)
    d = cp.causal_product_bwd_delta(*args(x), x["go"], ckpt, grad_state_out=x["gs"])
    a = [f64(t) for t in args(x)]
    r_out, r_s, _ = ref.delta_fwd(*a, 1.0, f64(x["s0"]))
    r_d = ref.delta_bwd(*a, 1.0, f64(x["go"]), f64(x["gs"]), f64(x["s0"]))
    close(out, r_out, "out")
    close(s, r_s, "state")
    for got, want, name in zip(d, r_d, ("dq", "dk", "dv", "dg", "dbeta")):
        close(got, want, name)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_nan_and_inf_stay_in_their_head(dt):
    x = make(1, 3, 3, 100, 64, 64, DT[dt], seed=8)
    clean = cp.causal_product_fwd_delta(*args(x))
    x["v"][0, 1, 70, 3], x["k"][0, 2, 80, 0] = float("nan"), float("inf")
    out, s = cp.causal_product_fwd_delta(*args(x), return_state=True)
    assert torch.equal(out[:, 0], clean[:, 0])
    assert torch.equal(out[:, 1:, :64], clean[:, 1:, :64])
    assert torch.isnan(out[0, 1, 70:, 3]).all() and torch.isnan(s[0, 1, :, 3]).any()
    assert not torch.isfinite(out[0, 2, 81:]).any()
    x["g"][0, 0, 50] = float("nan")
    out = cp.causal_product_fwd_delta(*args(x))
    assert torch.isnan(out[0, 0, 50:]).all()


@pytest.mark.parametrize("dt,D,M", [("bf16", 64, 64), ("bf16", 128, 128), ("f16", 64, 64)])
def test_pieces_of_a_sequence(dt, D, M):
    """A sequence in pieces, the state handed on, and its tokens one by one."""
    x = make(2, 2, 1, 170, D, M, DT[dt], seed=9, carry=True)
    r_out, r_s, _ = ref.delta_fwd(*[f64(t) for t in args(x)], 0.5, f64(x["s0"]))
    state, rows = x["s0"], []
    for lo, hi in ((0, 64), (64, 101), (101, 102)):
        piece = [t[:, :, lo:hi].contiguous() for t in args(x)]
        out, state = cp.causal_product_fwd_delta(*piece, state_in=state, return_state=True, scale=0.5)
        rows.append(out)
    for t in range(102, 170):
        row = cp.causal_product_decode_delta(*(y[:, :, t].contiguous() for y in args(x)), state,
                                             scale=0.5)
        rows.append(row[:, :, None])
    close(torch.cat(rows, 2), r_out, "out")
    close(state, r_s, "state")


@pytest.mark.parametrize("dt,N,D,M", [("bf16", 1500, 64, 64), ("bf16", 700, 128, 128),
                                      ("bf16", 2500, 64, 72)])
def test_long_sequences_agree_with_fp32(dt, N, D, M):
    """Long sequences against the CUDA-core path on the same values (held to
    the 64-bit recurrence above): twice the bound."""
    x = make(1, 2, 2, N, D, M, DT[dt], seed=10, carry=True, rate=0.02)
    y = {n: None if t is None else t.float() for n, t in x.items()}
    got, want = [], []
    for z, to in ((x, got), (y, want)):
        out, s, ckpt = cp.causal_product_fwd_delta(*args(z), state_in=z["s0"], return_state=True, save=True)
        to += [out, s, *cp.causal_product_bwd_delta(*args(z), z["go"], ckpt, grad_state_out=z["gs"],
                                                    return_state_grad=True)]
    for a, b in zip(got, want):
        assert err(a, f64(b)) <= TOL[a.dtype] + 1e-5


def test_gradients_against_differences():
    """Directional central differences of the fp32 forward.  With h = 1e-2 the
    h^2 term is ~1e-4 of the gradient and fp32 rounding 1e-7 |L| / h less."""
    x = make(1, 2, 1, 70, 32, 32, torch.float32, seed=11, carry=True)
    _, ckpt = cp.causal_product_fwd_delta(*args(x), state_in=x["s0"], save=True)
    d = cp.causal_product_bwd_delta(*args(x), x["go"], ckpt, grad_state_out=x["gs"],
                                    return_state_grad=True)

    def loss(y):
        out, s = cp.causal_product_fwd_delta(*args(y), state_in=y["s0"], return_state=True)
        return (out.double() * x["go"].double()).sum() + (s.double() * x["gs"].double()).sum()

    gen = torch.Generator(device=DEV).manual_seed(1)
    for name, grad in zip(("q", "k", "v", "g", "beta", "s0"), d):
        way = torch.randn(grad.shape, generator=gen, device=DEV)
        way = way / way.norm()
        h = 1e-2
        up = loss(dict(x, **{name: x[name] + h * way}))
        down = loss(dict(x, **{name: x[name] - h * way}))
        want = (grad.double() * way.double()).sum()
        assert abs((up - down) / (2 * h) - want) <= 2e-3 * grad.double().norm(), name


def test_autograd_and_no_grad():
    x = make(1, 4, 2, 90, 64, 64, torch.bfloat16, seed=12, carry=True)
    leaves = [t.clone().requires_grad_(True) for t in args(x) + [x["s0"]]]
    out, s = cp.causal_product_delta(*leaves[:5], state=leaves[5], return_state=True, scale=0.3)
    grads = torch.autograd.grad((out, s), leaves, (x["go"], x["gs"]))
    r = ref.delta_bwd(*[f64(t) for t in args(x)], 0.3, f64(x["go"]), f64(x["gs"]), f64(x["s0"]))
    for got, want in zip(grads, r):
        close(got, want)
    # only the state's gradient, and only the output's
    (gs,) = torch.autograd.grad(cp.causal_product_delta(*leaves[:5], leaves[5], True)[1].sum(), leaves[5])
    assert gs.shape == x["s0"].shape
    out1 = cp.causal_product_delta(*leaves[:5], state=leaves[5], scale=0.3)
    (gv,) = torch.autograd.grad(out1, leaves[2], x["go"])
    assert torch.equal(out1.detach(), out.detach()) and gv.shape == x["v"].shape
    with torch.no_grad():
        plain = cp.causal_product_delta(*leaves[:5], state=leaves[5], scale=0.3)
    assert torch.equal(plain, out.detach()) and not plain.requires_grad


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_repeatable_and_on_another_stream(dt):
    x = make(2, 4, 2, 300, 64, 128, DT[dt], seed=13, carry=True)

    def both(stream=None):
        out, s, ckpt = cp.causal_product_fwd_delta(*args(x), state_in=x["s0"], return_state=True,
                                                   save=True, stream=stream)
        return [out, s, *cp.causal_product_bwd_delta(*args(x), x["go"], ckpt, grad_state_out=x["gs"],
                                                     return_state_grad=True, stream=stream)]

    first = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = both()
        side.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_buffers_beside_the_outputs_stay(dt):
    """Outputs given as views of larger buffers: nothing outside is written,
    and a workspace of exactly the asked size does."""
    B, H, Hk, N, D, M = 1, 2, 1, 77, 64, 72
    x = make(B, H, Hk, N, D, M, DT[dt], seed=14, carry=True)
    pad = 1024

    def guarded(shape, dtype):
        n = int(np.prod(shape))
        buf = torch.full((n + 2 * pad,), 7.0, dtype=dtype, device=DEV)
        return buf, buf[pad:pad + n].view(shape)

    n_ck = cp.causal_product_delta_checkpoint_size(B, H, Hk, N, D, M, DT[dt]) // 4
    made = [guarded(s, t) for s, t in (((B, H, N, M), DT[dt]), ((B, H, D, M), torch.float32),
                                       ((n_ck,), torch.float32))]
    ws = [torch.zeros(cp.causal_product_delta_workspace_size(B, H, Hk, N, D, M, DT[dt], b),
                      dtype=torch.uint8, device=DEV) for b in (False, True)]
    cp.causal_product_fwd_delta(*args(x), out=made[0][1], state_in=x["s0"], return_state=True,
                                state_out=made[1][1], ckpt=made[2][1], workspace=ws[0])
    grads = [guarded(t.shape, t.dtype) for t in args(x)] + [guarded((B, H, D, M), torch.float32)]
    cp.causal_product_bwd_delta(*args(x), x["go"], made[2][1], *(g[1] for g in grads[:5]),
                                workspace=ws[1], grad_state_out=x["gs"], grad_state_in=grads[5][1],
                                return_state_grad=True)
    torch.cuda.synchronize()
    for buf, view in made + grads:
        assert (buf[:pad] == 7).all() and (buf[-pad:] == 7).all()
        assert torch.isfinite(view.float()).all()
    for w in ws:
        assert cp.causal_product_status(w) == cp.CP_OK
    a = [f64(t) for t in args(x)]
    close(made[0][1], ref.delta_fwd(*a, 1.0, f64(x["s0"]))[0])
    close(grads[0][1], ref.delta_bwd(*a, 1.0, f64(x["go"]), f64(x["gs"]), f64(x["s0"]))[0])


def test_no_rows():
    e = lambda *s: torch.empty(s, device=DEV)  # noqa: E731
    s0 = torch.randn(1, 2, 8, 8, device=DEV)
    x = (e(1, 2, 0, 8), e(1, 2, 0, 8), e(1, 2, 0, 8), e(1, 2, 0), e(1, 2, 0))
    out, s, ckpt = cp.causal_product_fwd_delta(*x, state_in=s0, return_state=True, save=True)
    assert out.shape == (1, 2, 0, 8) and torch.equal(s, s0)
    d = cp.causal_product_bwd_delta(*x, e(1, 2, 0, 8), ckpt, grad_state_out=s0, return_state_grad=True)
    assert torch.equal(d[5], s0)


# ------------------------------------------------------------------ decode
@pytest.mark.parametrize("shape", [(1, 16, 16, 64, 64, "bf16"), (7, 4, 2, 128, 128, "bf16"),
                                   (3, 2, 1, 40, 72, "bf16"), (2, 2, 2, 256, 256, "bf16"),
                                   (5, 3, 1, 64, 64, "f16"), (2, 2, 2, 65, 30, "f16"),
                                   (2, 2, 1, 16, 16, "f32"), (3, 1, 1, 7, 5, "f32"),
                                   (1, 1, 1, 256, 255, "f32"), (1, 1, 1, 1, 1, "f32"),
                                   # 256 MiB of states: the streaming variant
                                   (512, 16, 8, 64, 128, "bf16")],
                         ids=lambda s: "x".join(map(str, s)))
def test_decode_step(shape):
    B, H, Hk, D, M, dt = shape
    x = make(B, H, Hk, 1, D, M, DT[dt], seed=D + M, carry=True)
    state = x["s0"].clone()
    out = cp.causal_product_decode_delta(*(t[:, :, 0].contiguous() for t in args(x)), state, scale=0.4)
    r_out, r_s, _ = ref.delta_fwd(*[f64(t) for t in args(x)], 0.4, f64(x["s0"]))
    close(out, r_out[:, :, 0], "out")
    close(state, r_s, "state")


def test_decode_slots():
    """States of a pool: the named ones advance, the others stay; slots outside
    the pool are idle rows; a cleared state forgets NaN-free contents."""
    B, H, D, M, P = 6, 2, 64, 64, 9
    x = make(B, H, H, 1, D, M, torch.bfloat16, seed=3)
    pool = torch.randn(P, H, D, M, device=DEV)
    slots = torch.tensor([4, -1, 0, 8, 9, 2], dtype=torch.int32, device=DEV)
    x["g"][3] = -np.inf
    s0 = pool[slots.long().clamp(0, P - 1)]
    after = pool.clone()
    out = cp.causal_product_decode_delta(*(t[:, :, 0].contiguous() for t in args(x)), after, slots=slots)
    r_out, r_s, _ = ref.delta_fwd(*[f64(t) for t in args(x)], 1.0, f64(s0))
    live = [0, 2, 3, 5]
    close(out[live], r_out[live, :, 0])
    close(after[slots[live].long()], r_s[live])
    assert not out[[1, 4]].any()
    rest = [1, 3, 5, 6, 7]
    assert torch.equal(after[rest], pool[rest])


def test_decode_pool_past_32_bits():
    """A pool of more than 2^31 state elements, the last slot."""
    P, D, M = 32_900, 256, 256
    x = make(1, 1, 1, 1, D, M, torch.bfloat16, seed=4, carry=True)
    pool = torch.empty((P, 1, D, M), device=DEV)
    pool[P - 1] = x["s0"][0]
    out = cp.causal_product_decode_delta(*(t[:, :, 0].contiguous() for t in args(x)), pool,
                                         slots=torch.tensor([P - 1], dtype=torch.int32, device=DEV))
    r_out, r_s, _ = ref.delta_fwd(*[f64(t) for t in args(x)], 1.0, f64(x["s0"]))
    close(out, r_out[:, :, 0])
    close(pool[P - 1:], r_s)


def test_decode_in_a_graph():
    x = make(2, 4, 2, 1, 64, 64, torch.bfloat16, seed=15, carry=True)
    row = [t[:, :, 0].contiguous() for t in args(x)]
    state, want = x["s0"].clone(), x["s0"].clone()
    out = torch.empty(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    cp.causal_product_decode_delta(*row, state.clone(), out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cp.causal_product_decode_delta(*row, state, out=out)
    for _ in range(3):
        graph.replay()
        r = cp.causal_product_decode_delta(*row, want)
        assert torch.equal(out, r) and torch.equal(state, want)


# ---------------------------------------------------------------- refusals
def test_refusals():
    x = make(1, 2, 1, 20, 64, 64, torch.bfloat16, seed=16)
    q, k, v, g, b = args(x)
    fwd = cp.causal_product_fwd_delta
    with pytest.raises(ValueError):
        fwd(q, k[:, :, :10], v, g, b)                              # lengths differ
    with pytest.raises(ValueError):
        fwd(torch.cat([q] * 3, 1), torch.cat([k] * 3, 1), v, g, b)  # 3 key heads, 2 value heads
    with pytest.raises(ValueError):
        fwd(q, k, v, g.bfloat16(), b)                              # gates are float32
    with pytest.raises(ValueError):
        fwd(q, k, v, g, b[:, :1])
    with pytest.raises(TypeError):
        fwd(q, k.half(), v, g, b)
    with pytest.raises(ValueError):
        fwd(q, k, v.transpose(1, 2).contiguous().transpose(1, 2), g, b)
    with pytest.raises(RuntimeError):
        fwd(q, k, v, g.cpu(), b)
    with pytest.raises(ValueError):
        fwd(q, k, v, g, b, state_in=torch.zeros(1, 2, 64, 32, device=DEV))
    with pytest.raises(ValueError):
        fwd(q, k, v, g, b, ckpt=torch.zeros(8, device=DEV))
    with pytest.raises(cp.CausalProductError):
        fwd(q, k, v, g, b, scale=float("nan"))
    with pytest.raises(cp.CausalProductError):
        fwd(q, k, v, g, b, out=v)                                  # output over an input
    with pytest.raises(cp.CausalProductError):
        fwd(q, k, v, g, b, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(cp.CausalProductError):
        fwd(*(t[..., :60].contiguous() for t in (q, k, v)), g, b)  # rows of 120 bytes
    _, ckpt = fwd(q, k, v, g, b, save=True)
    with pytest.raises(ValueError):
        cp.causal_product_bwd_delta(q, k, v, g, b, x["go"][:, :, :5].contiguous(), ckpt)
    with pytest.raises(ValueError):
        cp.causal_product_bwd_delta(q, k, v, g, b, x["go"], None)
    with pytest.raises(ValueError):
        cp.causal_product_bwd_delta(q, k, v, g, b, x["go"], ckpt[:8].contiguous())
    with pytest.raises(cp.CausalProductError):
        cp.causal_product_bwd_delta(q, k, v, g, b, x["go"], ckpt, grad_v=v)
    row = [t[:, :, 0].contiguous() for t in (q, k, v, g, b)]
    state = torch.zeros(1, 2, 64, 64, device=DEV)
    dec = cp.causal_product_decode_delta
    with pytest.raises(ValueError):
        dec(*row, state[:0])
    with pytest.raises(ValueError):
        dec(*row, state.half())
    with pytest.raises(ValueError):
        dec(*row, state, slots=torch.zeros(1, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        dec(*row, state, slots=torch.zeros(2, dtype=torch.int32, device=DEV))
    with pytest.raises(cp.CausalProductError):
        dec(*row, state, out=row[2])
