"""The gated delta rule with slow decays that are the same at every token
(``-m gpu``), as a learned decay per head gives them: a state then remembers
thousands of tokens, and whatever a step's decay is off by adds up over them.

With nothing written (beta = 0) the state after N tokens is S_0 times the
product of the decays.  Every step rounds each element of the state once, by at
most 2^-24 of it and of random sign, so n steps leave at most sqrt(n) 2^-24 in
the 2-norm; the steps are tokens in decoding and at least 32 rows in a chunked
call.  A step's decay itself is held to far less than 2^-24; 4 x 2^-24 more is
for what a call rounds once."""
import numpy as np
import pytest
import torch

import prefix_sum_outer_gb300 as cp
from test_delta_gpu import DEV, DT, args, close, err, f64, make, ref

pytestmark = pytest.mark.gpu

RATES = (-1e-4, -1.017e-4, -1.37e-4, -3.3e-4, -1e-3, -4e-3)   # a head each


def slow(N, dt, beta, seed, D=64, M=32):
    H = len(RATES)
    x = make(1, H, H, N, D, M, DT[dt], seed=seed, carry=True)
    x["g"] = torch.tensor(RATES, device=DEV)[None, :, None].expand(1, H, N).contiguous()
    x["beta"] = torch.zeros_like(x["g"])
    x["beta"][..., ::7] = beta
    return x


def bound(steps):
    return (steps ** 0.5 + 4) * 2.0 ** -24


def kept(x, s):
    """S_0 (or a gradient) times the product of a head's decays, in 64 bits."""
    return f64(s) * np.exp(f64(x["g"]).sum(-1))[..., None, None]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_state_kept_over_a_long_sequence(dt):
    N = 8000
    x = slow(N, dt, 0.0, seed=31)
    _, s, ckpt = cp.causal_product_fwd_delta(*args(x), state_in=x["s0"], return_state=True, save=True)
    d = cp.causal_product_bwd_delta(*args(x), torch.zeros_like(x["go"]), ckpt, grad_state_out=x["gs"],
                                    return_state_grad=True)
    for h in range(len(RATES)):
        for got, want, name in ((s, kept(x, x["s0"]), "state"), (d[5], kept(x, x["gs"]), "dstate")):
            e = err(got[:, h], want[:, h])
            assert e <= bound(N / 32), f"{name}, g = {RATES[h]}: {e:.3g}"


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_state_kept_token_by_token(dt):
    N = 4096
    x = slow(1, dt, 0.0, seed=32)
    row = [t[:, :, 0].contiguous() for t in args(x)]
    state = x["s0"].clone()
    for _ in range(N):
        cp.causal_product_decode_delta(*row, state)
    want = f64(x["s0"]) * np.exp(N * f64(x["g"]))[..., None]
    for h in range(len(RATES)):
        e = err(state[:, h], want[:, h])
        assert e <= bound(N), f"g = {RATES[h]}: {e:.3g}"


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_writes_into_a_long_memory(dt):
    """Outputs, states and gradients with a write every seventh token."""
    x = slow(2500, dt, 0.05, seed=33)
    out, s, ckpt = cp.causal_product_fwd_delta(*args(x), state_in=x["s0"], return_state=True,
                                               scale=0.3, save=True)
    d = cp.causal_product_bwd_delta(*args(x), x["go"], ckpt, scale=0.3, grad_state_out=x["gs"],
                                    return_state_grad=True)
    a = [f64(t) for t in args(x)]
    r_out, r_s, _ = ref.delta_fwd(*a, 0.3, f64(x["s0"]))
    r_d = ref.delta_bwd(*a, 0.3, f64(x["go"]), f64(x["gs"]), f64(x["s0"]))
    for h in range(len(RATES)):
        close(out[:, h], r_out[:, h], "out")
        close(s[:, h], r_s[:, h], "state")
        for got, want, name in zip(d, r_d, ("dq", "dk", "dv", "dg", "dbeta", "dstate")):
            close(got[:, h], want[:, h], name)
