"""What the tensor cores cost linear attention with a decay in precision
(``-m gpu``): nothing beside fp32 arithmetic where a result is fp32, and less than
its own rounding where it is bf16.

Results in fp32 (the states, their gradients) are held to what the CUDA-core
kernels, fp32 throughout, leave on the same values: at most 1.5 times their error
against 64 bits, or 1e-6 (16 roundings of 2^-24) where that is more.

Results in bf16 are compared with the 64-bit ones rounded to bf16: where both
round to the same number nothing is left, and an error of e (relative to the
result's size, before rounding) moves an element of size x to the next one, u(x)
= 2^-8 to 2^-7 of it away, with probability |e| / u(x).  The squares' sum is u(x) |e|
per element, sqrt(0.0044 e) in the 2-norm.  P, the state's copy and, where no state
is asked for, the rows it takes enter their products as two bf16 numbers each, 2^-17
of an element at most, 2^-17 / sqrt(3) = 4.4e-6 of the whole and at most sqrt(2) of
that together (a result's two parts, P C and A S, have one or two such factors):
6.2e-6, so 1.65e-4.  The bound is 2e-4."""
import numpy as np
import pytest
import torch

from test_decay_gpu import DT, NAMES, err, f64, make, results, wanted

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [
    (2, 4, 2, 600, 64, 64), (1, 2, 1, 500, 128, 128), (1, 4, 2, 333, 96, 72), (2, 2, 2, 190, 40, 104),
    (1, 1, 1, 128 * 40 + 5, 64, 64), (1, 8, 1, 129, 128, 64), (1, 1, 1, 3000, 128, 128)],
    ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("rate", [-0.3, -0.01, 0.0])
def test_as_fp32(shape, rate):
    x = make(*shape, DT["bf16"], seed=sum(shape), carry=True, rates=[rate] * shape[1])
    got, want = results(x), wanted(x)
    fp32 = results({n: t if n in ("n", "g") or t is None else t.float() for n, t in x.items()})
    for n in NAMES:
        if got[n].dtype == torch.float32:
            e, most = err(got[n], want[n]), max(1e-6, 1.5 * err(fp32[n], want[n]))
        else:
            r = f64(torch.from_numpy(np.ascontiguousarray(want[n])).to(torch.bfloat16))
            e, most = err(got[n], r), 2e-4
        assert e <= most, f"{n}: {e:.3g} > {most:.3g}"
