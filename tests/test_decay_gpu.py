"""Linear attention with a decay for each head on the GPU (``-m gpu``): the
chunked forward and backward and the one-token step against the 64-bit
recurrence.

Errors are the 2-norm of the difference over the 2-norm of the result.  Bounds,
set by the arithmetic: results in fp32 are at most 2e-6 off, 32 roundings of
2^-24, for their sums have a few hundred products of random sign (an error of
about sqrt(300) / 2 roundings of the partial sums) and their powers of the decay a
few roundings each; a result rounded once to bf16 (8 significant bits) is at most
2^-8 = 3.9e-3 off, to fp16 (11 bits) 2^-11 = 4.9e-4, and on the way there a
factor held as two bf16 numbers (16 bits) leaves at most 2^-17 = 7.6e-6."""
import numpy as np
import pytest
import torch

import decay_reference as ref
import prefix_sum_outer_gb300 as cp

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TOL = {torch.bfloat16: 2.0 ** -8 + 1e-5, torch.float16: 2.0 ** -11 + 1e-5, torch.float32: 2e-6}
NAMES = ("out", "state", "dq", "dk", "dv", "dstate")


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


def make(B, H, Hk, N, D, M, dt, seed, carry=False, rates=None, lengths=None):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    if rates is None:  # memories of a token to some hundreds
        rates = -torch.exp(torch.rand((H,), generator=gen) * 7 - 6)
    x = {"q": rnd(B, Hk, N, D).to(dt), "k": (rnd(B, Hk, N, D) + 0.5 * rnd(1, Hk, 1, D)).to(dt),
         "v": rnd(B, H, N, M).to(dt), "g": torch.as_tensor(rates, dtype=torch.float32),
         "go": rnd(B, H, N, M).to(dt), "s0": rnd(B, H, D, M) if carry else None,
         "gs": rnd(B, H, D, M) if carry else None,
         "n": None if lengths is None else torch.tensor(lengths, dtype=torch.int32)}
    return {n: None if t is None else t.to(DEV) for n, t in x.items()}


def args(x):
    return [x[n] for n in ("q", "k", "v", "g")]


def results(x, scale=0.3, stream=None):
    kw = dict(scale=scale, lengths=x["n"], stream=stream)
    out, s = cp.causal_product_fwd_decay(*args(x), state_in=x["s0"], return_state=True, **kw)
    d = cp.causal_product_bwd_decay(*args(x), x["go"], state_in=x["s0"], grad_state_out=x["gs"],
                                    return_state_grad=True, **kw)
    return dict(zip(NAMES, (out, s, *d)))


def wanted(x, scale=0.3):
    a = [f64(t) for t in args(x)]
    a[3] = np.maximum(a[3], -120.0)
    s0, gs, n = f64(x["s0"]), f64(x["gs"]), None if x["n"] is None else x["n"].cpu().numpy()
    out, s, _ = ref.decay_fwd(*a, scale, s0, n)
    return dict(zip(NAMES, (out, s, *ref.decay_bwd(*a, scale, f64(x["go"]), gs, s0, n))))


def check(x, scale=0.3):
    got, want = results(x, scale), wanted(x, scale)
    plain = cp.causal_product_fwd_decay(*args(x), state_in=x["s0"], scale=scale, lengths=x["n"])
    grads = cp.causal_product_bwd_decay(*args(x), x["go"], state_in=x["s0"],
                                        grad_state_out=x["gs"], scale=scale, lengths=x["n"])
    torch.cuda.synchronize()
    for n in NAMES:
        close(got[n], want[n], n)
    # without the states asked for, to the same bounds
    for n, t in zip(("out", "dq", "dk", "dv"), (plain, *grads)):
        close(t, want[n], n)
    return got


# B, H, Hk, N, D, M, dtype, carried state
SHAPES = [
    (1, 1, 1, 1, 8, 8, "bf16", False), (2, 2, 1, 1, 64, 64, "bf16", True),
    (1, 2, 2, 63, 64, 64, "bf16", False), (1, 2, 2, 64, 64, 64, "bf16", True),
    (1, 2, 1, 65, 64, 64, "bf16", True), (1, 2, 2, 127, 64, 64, "bf16", True),
    (1, 2, 2, 128, 64, 64, "bf16", True), (1, 2, 2, 129, 64, 64, "bf16", True),
    (1, 2, 2, 200, 64, 128, "bf16", False), (1, 2, 2, 150, 128, 64, "bf16", True),
    (1, 4, 1, 257, 128, 128, "bf16", True), (1, 2, 2, 97, 40, 72, "bf16", True),
    (1, 1, 1, 130, 96, 16, "bf16", True), (2, 6, 3, 300, 72, 104, "bf16", True),
    (1, 1, 1, 70, 16, 200, "bf16", True), (1, 1, 1, 40, 256, 64, "bf16", True),
    (3, 40, 20, 260, 64, 64, "bf16", True),
    (2, 2, 2, 33, 64, 64, "f32", True), (1, 4, 2, 70, 64, 128, "f32", True),
    (1, 1, 1, 37, 5, 3, "f32", True), (1, 1, 1, 130, 256, 40, "f32", True),
    (1, 2, 2, 600, 33, 65, "f32", True), (2, 3, 1, 1, 16, 16, "f32", True),
    (1, 3, 3, 65, 64, 64, "f16", True), (1, 2, 1, 40, 72, 24, "f16", False),
    (1, 4, 4, 129, 128, 66, "f16", True), (1, 1, 1, 64, 1, 1, "f32", True),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward_and_backward(shape):
    B, H, Hk, N, D, M, dt, carry = shape
    check(make(B, H, Hk, N, D, M, DT[dt], seed=N + D + M, carry=carry))


# rates of no decay, of memories of ten thousand tokens to less than one, and none
RATES = (0.0, -1e-4, -0.01, -0.3, -3.0, -20.0, -119.0, -1e9, -np.inf)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N", [1, 100, 420])
def test_rates(dt, N):
    H = len(RATES)
    got = check(make(1, H, H, N, 64, 64, DT[dt], seed=6, carry=True, rates=RATES))
    # the token alone
    assert not got["dstate"][:, -2:].any()


@pytest.mark.parametrize("dt,D,M", [("bf16", 64, 64), ("bf16", 128, 128), ("bf16", 40, 72),
                                    ("f16", 64, 64), ("f32", 33, 64)])
def test_lengths(dt, D, M):
    """A padded batch: rows behind a sequence's end reach nothing, NaN and inf
    among them, and give zero; lengths outside [0, N] are taken into it."""
    n, N = [0, 1, 64, 127, 128, 129, 300, 256, 301, 77], 301
    x = make(len(n), 4, 2, N, D, M, DT[dt], seed=16, carry=True, lengths=n)
    for b, e in enumerate(n):
        for t in ("q", "k", "v", "go"):
            x[t][b, :, e:] = float("nan")
            x[t][b, :, e + 1::3] = float("inf")
    got = check(x)
    for b, e in enumerate(n):
        for t in ("out", "dq", "dk", "dv"):
            assert not got[t][b, :, e:].any()
    assert torch.equal(got["state"][0], x["s0"][0]) and torch.equal(got["dstate"][0], x["gs"][0])
    y = dict(x, n=torch.tensor([-5] + n[1:8] + [400, 77], dtype=torch.int32, device=DEV))
    again = results(y)
    for t in NAMES:
        assert torch.equal(again[t], got[t])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_nan_and_inf_stay_in_their_head(dt):
    x = make(1, 4, 4, 300, 64, 64, DT[dt], seed=8, rates=[-0.01] * 4)
    clean, _ = cp.causal_product_fwd_decay(*args(x), return_state=True)
    x["v"][0, 1, 140, 3], x["k"][0, 2, 180, 0] = float("nan"), float("inf")
    x["g"][3] = float("nan")
    out, s = cp.causal_product_fwd_decay(*args(x), return_state=True)
    assert torch.equal(out[:, 0], clean[:, 0])
    assert torch.equal(out[:, 1:3, :128], clean[:, 1:3, :128])
    assert torch.isnan(out[0, 1, 140:, 3]).all() and torch.isnan(s[0, 1, :, 3]).any()
    assert not torch.isfinite(out[0, 2, 181:]).any()
    assert torch.isnan(out[0, 3]).all() and torch.isnan(s[0, 3]).all()
    # a decay that would grow is no decay
    x["g"][0] = 1e-3
    d = results(x)
    for n in ("out", "dq", "dk", "dv"):
        assert torch.isnan(d[n][0, 0]).all(), n


@pytest.mark.parametrize("dt,D,M", [("bf16", 64, 64), ("bf16", 128, 128), ("f16", 64, 64)])
def test_pieces_of_a_sequence(dt, D, M):
    """A sequence in pieces, the state handed on, and its tokens one by one."""
    x = make(2, 2, 1, 300, D, M, DT[dt], seed=9, carry=True)
    r_out, r_s, _ = ref.decay_fwd(*[f64(t) for t in args(x)], 0.5, f64(x["s0"]))
    state, rows = x["s0"], []
    for lo, hi in ((0, 128), (128, 201), (201, 202)):
        piece = [t[:, :, lo:hi].contiguous() for t in args(x)[:3]] + [x["g"]]
        out, state = cp.causal_product_fwd_decay(*piece, state_in=state, return_state=True, scale=0.5)
        rows.append(out)
    for t in range(202, 300):
        row = cp.causal_product_decode_decay(*(y[:, :, t].contiguous() for y in args(x)[:3]), x["g"],
                                             state, scale=0.5)
        rows.append(row[:, :, None])
    close(torch.cat(rows, 2), r_out, "out")
    close(state, r_s, "state")


@pytest.mark.parametrize("dt,N,D,M", [("bf16", 1500, 64, 64), ("bf16", 2700, 128, 128),
                                      ("bf16", 6000, 64, 72), ("f16", 5000, 64, 64)])
def test_long_sequences_agree_with_fp32(dt, N, D, M):
    """Long sequences of few heads against the fp32 path on the same values
    (held to the 64-bit recurrence above): twice the bound."""
    x = make(1, 2, 2, N, D, M, DT[dt], seed=10, carry=True, rates=[-0.002, 0.0], lengths=[N - 5])
    y = {n: t if n in ("n", "g") or t is None else t.float() for n, t in x.items()}
    got, want = results(x), results(y)
    for n in NAMES:
        assert err(got[n], f64(want[n])) <= TOL[got[n].dtype] + 2e-6, n


def test_gradients_against_differences():
    """Directional differences of the fp32 forward, which is linear in each
    argument: rounding, 1e-6 of L, over h = 1."""
    x = make(1, 2, 1, 130, 32, 32, torch.float32, seed=11, carry=True)
    got = results(x)

    def loss(y):
        out, s = cp.causal_product_fwd_decay(*args(y), state_in=y["s0"], return_state=True, scale=0.3)
        return (out.double() * x["go"].double()).sum() + (s.double() * x["gs"].double()).sum()

    gen = torch.Generator(device=DEV).manual_seed(1)
    size = wanted(x)["out"]
    size = np.linalg.norm(size) * np.linalg.norm(f64(x["go"]))
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("s0", "dstate")):
        way = torch.randn(x[name].shape, generator=gen, device=DEV)
        slope = (loss(dict(x, **{name: x[name] + way})) - loss(dict(x, **{name: x[name] - way}))) / 2
        want = (got[grad].double() * way.double()).sum()
        assert abs(slope - want) <= 4e-6 * size, name


def test_autograd_and_no_grad():
    x = make(2, 4, 2, 190, 64, 64, torch.bfloat16, seed=12, carry=True, lengths=[190, 100])
    leaves = [x[n].clone().requires_grad_(True) for n in ("q", "k", "v", "s0")]
    q, k, v, s0 = leaves
    call = lambda **kw: cp.causal_product_decay(q, k, v, x["g"], state=s0, scale=0.3,  # noqa: E731
                                                lengths=x["n"], **kw)
    out, s = call(return_state=True)
    grads = torch.autograd.grad((out, s), leaves, (x["go"], x["gs"]))
    want = wanted(x)
    for got, n in zip(grads, ("dq", "dk", "dv", "dstate")):
        close(got, want[n], n)
    # only the state's gradient, and only the output's
    (gs,) = torch.autograd.grad(call(return_state=True)[1].sum(), s0)
    assert gs.shape == x["s0"].shape
    (gv,) = torch.autograd.grad(call(), v, x["go"])
    assert gv.shape == x["v"].shape
    # non-contiguous inputs and gradients
    odd = [t.detach().transpose(1, 2).contiguous().transpose(1, 2).requires_grad_(True)
           for t in (q, k, v)]
    out2 = cp.causal_product_decay(*odd, x["g"], state=x["s0"], scale=0.3, lengths=x["n"])
    d2 = torch.autograd.grad(out2, odd, x["go"].transpose(2, 3).contiguous().transpose(2, 3))
    d1 = torch.autograd.grad(call(), (q, k, v), x["go"])
    for a, b in zip(d1, d2):
        assert torch.equal(a, b)
    with torch.no_grad():
        plain = call()
    close(plain, want["out"])
    assert not plain.requires_grad
    with pytest.raises(ValueError):
        cp.causal_product_decay(q, k, v, x["g"].clone().requires_grad_(True))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_repeatable_and_on_another_stream(dt):
    x = make(2, 4, 2, 1100, 64, 128, DT[dt], seed=13, carry=True, lengths=[1100, 700])
    first = results(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = results(x)
        side.synchronize()
    third = results(x, stream=side)
    side.synchronize()
    for n in NAMES:
        assert torch.equal(first[n], second[n]) and torch.equal(first[n], third[n])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [77, 1030])
def test_buffers_beside_the_outputs_stay(dt, N):
    """Outputs given as views of larger buffers: nothing outside is written,
    and a workspace of exactly the asked size does."""
    B, H, Hk, D, M = 1, 2, 1, 64, 72
    x = make(B, H, Hk, N, D, M, DT[dt], seed=14, carry=True)
    pad = 1024

    def guarded(shape, dtype):
        n = int(np.prod(shape))
        buf = torch.full((n + 2 * pad,), 7.0, dtype=dtype, device=DEV)
        return buf, buf[pad:pad + n].view(shape)

    made = [guarded(s, t) for s, t in (((B, H, N, M), DT[dt]), ((B, H, D, M), torch.float32))]
    spaces = []
    for back in (False, True):
        n = cp.causal_product_decay_workspace_size(B, H, Hk, N, D, M, DT[dt], back)
        buf = torch.full((n + 256,), 7, dtype=torch.uint8, device=DEV)
        buf[:256] = 0
        spaces.append((buf, buf[:n]))
    cp.causal_product_fwd_decay(*args(x), out=made[0][1], state_in=x["s0"], return_state=True,
                                state_out=made[1][1], workspace=spaces[0][1])
    grads = [guarded(t.shape, t.dtype) for t in args(x)[:3]] + [guarded((B, H, D, M), torch.float32)]
    cp.causal_product_bwd_decay(*args(x), x["go"], *(g[1] for g in grads[:3]), workspace=spaces[1][1],
                                state_in=x["s0"], grad_state_out=x["gs"], grad_state_in=grads[3][1],
                                return_state_grad=True)
    torch.cuda.synchronize()
    for buf, view in made + grads:
        assert (buf[:pad] == 7).all() and (buf[-pad:] == 7).all()
        assert torch.isfinite(view.float()).all()
    for buf, ws in spaces:
        assert cp.causal_product_status(ws) == cp.CP_OK and (buf[-256:] == 7).all()
    want = wanted(x, 1.0)
    for n, (_, view) in zip(NAMES, made + grads):
        close(view, want[n], n)


def test_no_rows():
    e = torch.empty((1, 2, 0, 8), device=DEV)
    g = torch.zeros(2, device=DEV)
    s0 = torch.randn(1, 2, 8, 8, device=DEV)
    out, s = cp.causal_product_fwd_decay(e, e, e, g, state_in=s0, return_state=True)
    assert out.shape == (1, 2, 0, 8) and torch.equal(s, s0)
    d = cp.causal_product_bwd_decay(e, e, e, g, e, grad_state_out=s0, return_state_grad=True)
    assert torch.equal(d[3], s0)


def test_without_decay_it_is_the_causal_product():
    """log_decay = 0 against the framework's own causal product."""
    x = make(2, 3, 3, 500, 64, 64, torch.bfloat16, seed=17, rates=[0.0] * 3)
    got = cp.causal_product_fwd_decay(*args(x))
    want = cp.causal_product_fwd(x["q"], x["k"], x["v"])
    # both are rounded once, each by at most 2^-8
    assert err(got, f64(want)) <= 2 * TOL[torch.bfloat16]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_graphs(dt):
    """Forward and backward captured and replayed on new inputs, two graphs in
    one memory pool and on one workspace."""
    x = make(1, 2, 2, 700, 64, 64, DT[dt], seed=18, carry=True)
    y = make(1, 2, 2, 700, 64, 64, DT[dt], seed=19, carry=True)
    dims = (1, 2, 2, 700, 64, 64, DT[dt])
    ws = torch.zeros(max(cp.causal_product_decay_workspace_size(*dims, b) for b in (False, True)),
                     dtype=torch.uint8, device=DEV)

    def run():
        out, s = cp.causal_product_fwd_decay(*args(x), state_in=x["s0"], return_state=True, workspace=ws)
        return [out, s, *cp.causal_product_bwd_decay(*args(x), x["go"], state_in=x["s0"], workspace=ws,
                                                     grad_state_out=x["gs"], return_state_grad=True)]

    run()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=graphs[0][0].pool() if graphs else None):
            graphs.append((g, run()))
    for n in ("q", "k", "v", "go", "s0", "gs"):
        x[n].copy_(y[n])
    x["g"].copy_(y["g"])
    want = [t.clone() for t in run()]
    for g, got in graphs:
        g.replay()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


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
    row = [t[:, :, 0].contiguous() for t in args(x)[:3]] + [x["g"]]
    out = cp.causal_product_decode_decay(*row, state, scale=0.4)
    r_out, r_s, _ = ref.decay_fwd(*[f64(t) for t in args(x)], 0.4, f64(x["s0"]))
    close(out, r_out[:, :, 0], "out")
    close(state, r_s, "state")


def test_decode_slots():
    """States of a pool: the named ones advance, the others stay; slots outside
    the pool are idle rows; a head without memory keeps the token alone."""
    B, H, D, M, P = 6, 2, 64, 64, 9
    x = make(B, H, H, 1, D, M, torch.bfloat16, seed=3, rates=[-0.1, -np.inf])
    pool = torch.randn(P, H, D, M, device=DEV)
    slots = torch.tensor([4, -1, 0, 8, 9, 2], dtype=torch.int32, device=DEV)
    s0 = pool[slots.long().clamp(0, P - 1)]
    after = pool.clone()
    row = [t[:, :, 0].contiguous() for t in args(x)[:3]] + [x["g"]]
    out = cp.causal_product_decode_decay(*row, after, slots=slots)
    a = [f64(t) for t in args(x)]
    r_out, r_s, _ = ref.decay_fwd(*a, 1.0, f64(s0))
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
    row = [t[:, :, 0].contiguous() for t in args(x)[:3]] + [x["g"]]
    out = cp.causal_product_decode_decay(*row, pool,
                                         slots=torch.tensor([P - 1], dtype=torch.int32, device=DEV))
    r_out, r_s, _ = ref.decay_fwd(*[f64(t) for t in args(x)], 1.0, f64(x["s0"]))
    close(out, r_out[:, :, 0])
    close(pool[P - 1:], r_s)


def test_decode_in_a_graph():
    x = make(2, 4, 2, 1, 64, 64, torch.bfloat16, seed=15, carry=True)
    row = [t[:, :, 0].contiguous() for t in args(x)[:3]] + [x["g"]]
    state, want = x["s0"].clone(), x["s0"].clone()
    out = torch.empty(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    cp.causal_product_decode_decay(*row, state.clone(), out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cp.causal_product_decode_decay(*row, state, out=out)
    for _ in range(3):
        graph.replay()
        r = cp.causal_product_decode_decay(*row, want)
        assert torch.equal(out, r) and torch.equal(state, want)


# ------------------------------------------------------------- slow decays
SLOW = (-1e-4, -1.017e-4, -1.37e-4, -3.3e-4, -1e-3, -4e-3)   # a head each


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_state_kept_over_a_long_sequence(dt):
    """With nothing written (k = 0, q = 0) the state after n tokens is S_0 times
    e^{g n}, and so is the gradient: each step rounds each element once, by at
    most 2^-24 of random sign, sqrt(steps) 2^-24 in the 2-norm, a step being a
    token in decoding and at least 64 rows in a chunked call; 4 x 2^-24 more is
    for what a call rounds once."""
    N, H = 8000, len(SLOW)
    x = make(1, H, H, N, 64, 32, DT[dt], seed=31, carry=True, rates=SLOW)
    x["k"].zero_(), x["q"].zero_()
    got = results(x)
    state = x["s0"].clone()
    row = [t[:, :, 0].contiguous() for t in args(x)[:3]] + [x["g"]]
    for _ in range(4096):
        cp.causal_product_decode_decay(*row, state)
    kept = lambda t, n: f64(t) * np.exp(f64(x["g"]) * n)[:, None, None]  # noqa: E731
    for h in range(H):
        for a, w, steps in ((got["state"], kept(x["s0"], N), N / 64),
                            (got["dstate"], kept(x["gs"], N), N / 64),
                            (state, kept(x["s0"], 4096), 4096)):
            assert err(a[:, h], w[:, h]) <= (steps ** 0.5 + 4) * 2.0 ** -24


# ---------------------------------------------------------------- refusals
def test_refusals():
    x = make(1, 2, 1, 20, 64, 64, torch.bfloat16, seed=16)
    q, k, v, g = args(x)
    fwd = cp.causal_product_fwd_decay
    with pytest.raises(ValueError):
        fwd(q, k[:, :, :10], v, g)                              # lengths differ
    with pytest.raises(ValueError):
        fwd(torch.cat([q] * 3, 1), torch.cat([k] * 3, 1), v, g)  # 3 key heads, 2 value heads
    with pytest.raises(ValueError):
        fwd(q, k, v, g.bfloat16())                              # the decay is float32
    with pytest.raises(ValueError):
        fwd(q, k, v, g[:1])
    with pytest.raises(TypeError):
        fwd(q, k.half(), v, g)
    with pytest.raises(ValueError):
        fwd(q, k, v.transpose(1, 2).contiguous().transpose(1, 2), g)
    with pytest.raises(RuntimeError):
        fwd(q, k, v, g.cpu())
    with pytest.raises(RuntimeError):
        fwd(q, k, v, g, lengths=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        fwd(q, k, v, g, lengths=torch.zeros(1, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        fwd(q, k, v, g, state_in=torch.zeros(1, 2, 64, 32, device=DEV))
    with pytest.raises(cp.CausalProductError):
        fwd(q, k, v, g, scale=float("nan"))
    with pytest.raises(cp.CausalProductError):
        fwd(q, k, v, g, out=v)                                  # output over an input
    with pytest.raises(cp.CausalProductError):
        fwd(q, k, v, g, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(cp.CausalProductError):
        fwd(*(t[..., :60].contiguous() for t in (q, k, v)), g)  # rows of 120 bytes
    with pytest.raises(ValueError):
        cp.causal_product_bwd_decay(q, k, v, g, x["go"][:, :, :5].contiguous())
    with pytest.raises(cp.CausalProductError):
        cp.causal_product_bwd_decay(q, k, v, g, x["go"], grad_v=v)
    row = [t[:, :, 0].contiguous() for t in (q, k, v)] + [g]
    state = torch.zeros(1, 2, 64, 64, device=DEV)
    dec = cp.causal_product_decode_decay
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
