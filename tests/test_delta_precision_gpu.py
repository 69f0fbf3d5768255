"""What the tensor cores cost the gated delta rule in precision (``-m gpu``):
nothing beside fp32 arithmetic.

Results in fp32 (the carried state, its gradient, the gates' gradients) are held
to what the CUDA-core kernels, fp32 throughout, leave on the same values: at most
1.5 times their error against 64 bits, or 1e-6 (16 roundings of 2^-24) where that
is more.

Results in bf16 are compared with the 64-bit ones rounded to bf16: where both
round to the same number nothing is left, and an error of e (relative to the
result's size, before rounding) moves an element of size x to the next one, u(x)
= 2^-8 to 2^-7 of it away, with probability |e| / u(x).  The squares' sum is u(x) |e|
per element, 0.0055 x 0.8 e in the mean over normal x and e: sqrt(0.0044 e), 7e-5
at e = 1e-6, 1.5e-4 at the 5e-6 of factors held in 16 bits.  The bound is 1e-4."""
import numpy as np
import pytest
import torch

import prefix_sum_outer_gb300 as cp
from test_delta_gpu import DT, args, err, f64, make, ref

pytestmark = pytest.mark.gpu

NAMES = ("out", "state", "dq", "dk", "dv", "dg", "dbeta", "dstate")


def results(x, scale):
    out, s, ckpt = cp.causal_product_fwd_delta(*args(x), state_in=x["s0"], return_state=True,
                                               scale=scale, save=True)
    d = cp.causal_product_bwd_delta(*args(x), x["go"], ckpt, scale=scale, grad_state_out=x["gs"],
                                    return_state_grad=True)
    return dict(zip(NAMES, (out, s, *d)))


def wanted(x, scale):
    a = [f64(t) for t in args(x)]
    out, s, _ = ref.delta_fwd(*a, scale, f64(x["s0"]))
    return dict(zip(NAMES, (out, s, *ref.delta_bwd(*a, scale, f64(x["go"]), f64(x["gs"]), f64(x["s0"])))))


def check(x, scale=0.3, rounded=True):
    got, want = results(x, scale), wanted(x, scale)
    fp32 = results({n: None if t is None else t.float() for n, t in x.items()}, scale)
    for n in NAMES:
        if got[n].dtype == torch.float32:
            e, most = err(got[n], want[n]), max(1e-6, 1.5 * err(fp32[n], want[n]))
        elif rounded:
            r = f64(torch.from_numpy(np.ascontiguousarray(want[n])).to(torch.bfloat16))
            e, most = err(got[n], r), 1e-4
        else:
            continue
        assert e <= most, f"{n}: {e:.3g} > {most:.3g}"


@pytest.mark.parametrize("shape", [
    (2, 4, 2, 600, 64, 64), (1, 2, 1, 500, 128, 128), (1, 4, 2, 333, 96, 72), (1, 2, 2, 190, 40, 200),
    (1, 1, 1, 64 * 70 + 5, 64, 64), (1, 8, 1, 65, 128, 64)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("rate", [0.3, 0.01])
def test_as_fp32(shape, rate):
    check(make(*shape, DT["bf16"], seed=sum(shape), carry=True, rate=rate))


def test_repeated_keys():
    """Keys that all but coincide, at full strength and without decay."""
    x = make(1, 2, 2, 190, 64, 64, DT["bf16"], seed=41, carry=True, common=4.0, rate=0.0)
    x["beta"].fill_(1.0)
    check(x, rounded=False)
