"""How the factors of linear attention with a decay enter the tensor cores
(``-m gpu``): what else a call is asked for changes no bit of a result, and the
state and the rows that it takes are held in all of fp32's bits.

The bound of the second test.  Results in bf16 are compared with the 64-bit ones
rounded to bf16: an error e of an element of size x before rounding moves it to
the next number, u(x) = 2^-8 to 2^-7 of it away, with probability |e| / u(x), so the
2-norm of the difference is sqrt(0.0044 mean|e|) of the result's.  P alone is
rounded to two bf16 numbers: the first leaves a rest that is uniform in +-2^-8 of
the number's power of two, whose own rounding is 0.44 * 2^-17 of that (the mean square
over the rest's binades), 2.2e-6 of a score in the root mean square.  With a decay of
e^-0.001 a token a row reads, beside its tile (64 rows on average), the state of
hundreds before it, five times as many or more at all but the first tiles: P carries
at most 0.5 of the result in the 2-norm, mean|e| = 0.8 * 0.5 * 2.2e-6 = 9e-7.  The
accumulators' rounding toward zero adds 8 steps of 2^-24, 5e-7 at most.  In all
1.4e-6, and sqrt(0.0044 * 1.4e-6) = 7.8e-5.  With the state and its rows as two bf16
numbers as well it would be mean|e| = 0.8 * sqrt(2) * 2.2e-6 = 2.5e-6, 1.05e-4.

A call of one tile has its scores in three bf16 numbers, in full: what is left is the
rounding toward zero, 8 steps of 2^-24 in a score and as many in its product, 1e-6 at
most, sqrt(0.0044 * 1e-6) = 6.6e-5; with two numbers it would be 0.8 * 2.2e-6, 8.8e-5."""
import numpy as np
import pytest
import torch

import prefix_sum_outer_gb300 as cp
from test_decay_gpu import DT, args, err, f64, make, wanted

pytestmark = pytest.mark.gpu


def without_states(x, scale=0.3):
    kw = dict(state_in=x["s0"], scale=scale, lengths=x["n"])
    return (cp.causal_product_fwd_decay(*args(x), **kw),
            *cp.causal_product_bwd_decay(*args(x), x["go"], grad_state_out=x["gs"], **kw))


def with_states(x, scale=0.3):
    kw = dict(state_in=x["s0"], scale=scale, lengths=x["n"])
    out, _ = cp.causal_product_fwd_decay(*args(x), return_state=True, **kw)
    return (out, *cp.causal_product_bwd_decay(*args(x), x["go"], grad_state_out=x["gs"],
                                              return_state_grad=True, **kw)[:3])


@pytest.mark.parametrize("dt,shape,lengths", [
    ("bf16", (2, 4, 4, 700, 64, 64), [700, 333]), ("bf16", (1, 4, 2, 1500, 128, 128), None),
    ("bf16", (1, 2, 2, 900, 64, 128), None), ("bf16", (2, 4, 1, 300, 128, 40), [300, 129]),
    ("bf16", (3, 40, 40, 260, 64, 64), None), ("bf16", (1, 2, 1, 100, 72, 64), None),
    ("f16", (2, 4, 2, 300, 64, 64), [0, 257]), ("f32", (2, 4, 2, 300, 33, 40), [300, 64])])
def test_asking_for_a_state_changes_no_other_result(dt, shape, lengths):
    x = make(*shape, DT[dt], seed=61, carry=True, lengths=lengths)
    for name, a, b in zip(("out", "dq", "dk", "dv"), without_states(x), with_states(x)):
        assert torch.equal(a, b), name


@pytest.mark.parametrize("shape", [(1, 4, 4, 2500, 64, 64), (1, 2, 1, 2000, 128, 128)],
                         ids=lambda s: "x".join(map(str, s)))
def test_the_state_enters_in_full(shape):
    x = make(*shape, DT["bf16"], seed=62, carry=True, rates=[-0.001] * shape[1])
    want = wanted(x)
    for name, got in zip(("out", "dq", "dk", "dv"), without_states(x)):
        r = f64(torch.from_numpy(np.ascontiguousarray(want[name])).to(torch.bfloat16))
        assert err(got, r) <= 7.8e-5, f"{name}: {err(got, r):.3g}"


@pytest.mark.parametrize("shape", [(32, 8, 8, 100, 64, 64), (16, 4, 4, 128, 128, 128), (64, 8, 4, 17, 96, 72),
                                   (128, 8, 8, 3, 64, 64)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("carry", [False, True])
def test_one_tile_is_held_in_full(shape, carry):
    x = make(*shape, DT["bf16"], seed=63, carry=carry)
    want = wanted(x)
    for name, got in zip(("out", "dq", "dk", "dv"), without_states(x)):
        r = f64(torch.from_numpy(np.ascontiguousarray(want[name])).to(torch.bfloat16))
        assert err(got, r) <= 6.6e-5, f"{name}: {err(got, r):.3g}"
