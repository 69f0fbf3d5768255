"""The gated delta rule and the q/k norm on the GPU (``-m gpu``) where the other
tests' bounds leave room: what the fp32 kernels leave, and roundings to 16 bits.

fp32 results of the CUDA-core kernels: sums of up to a few hundred fp32
products, each step's rounding at most 2^-24 and of random sign; 16 of them, 1e-6.

16-bit results against the 64-bit ones rounded alike (test_delta_precision_gpu.py
has the derivation): sqrt(0.0044 e) for bf16 and, its steps being an eighth,
sqrt(0.00055 e) for fp16, at e = 1e-6 7e-5 and 2.4e-5; half as much again."""
import numpy as np
import pytest
import torch

import delta_reference as ref
import prefix_sum_outer_gb300 as cp
import test_qk_rope_gpu as rope
from test_delta_gpu import DT, args, err, f64, make
from test_delta_precision_gpu import NAMES, results, wanted

pytestmark = pytest.mark.gpu

MOST = {torch.float32: 1e-6, torch.bfloat16: 1e-4, torch.float16: 3.6e-5}


def near(got, want, name):
    if got.dtype != torch.float32:
        want = f64(torch.from_numpy(np.ascontiguousarray(want)).to(got.dtype))
    e = err(got, want)
    assert e <= MOST[got.dtype], f"{name}: {e:.3g}"


@pytest.mark.parametrize("shape", [
    (2, 4, 2, 300, 64, 64, "f32"), (1, 2, 1, 250, 128, 72, "f32"), (1, 1, 1, 150, 256, 40, "f32"),
    (1, 2, 2, 101, 31, 17, "f32"), (1, 4, 2, 300, 64, 64, "f16"), (1, 2, 1, 200, 200, 64, "bf16")],
    ids=lambda s: "x".join(map(str, s)))
def test_cuda_cores(shape):
    *dims, dt = shape
    x = make(*dims, DT[dt], seed=sum(dims), carry=True)
    got, want = results(x, 0.3), wanted(x, 0.3)
    for n in NAMES:
        near(got[n], want[n], n)


@pytest.mark.parametrize("shape", [(4, 4, 2, 128, 64, "bf16"), (9, 2, 1, 64, 64, "f16"), (5, 2, 2, 256, 40, "f32")],
                         ids=lambda s: "x".join(map(str, s)))
def test_one_token(shape):
    B, H, Hk, D, M, dt = shape
    x = make(B, H, Hk, 1, D, M, DT[dt], seed=D + M, carry=True)
    state = x["s0"].clone()
    out = cp.causal_product_decode_delta(*(t[:, :, 0].contiguous() for t in args(x)), state, scale=0.4)
    r_out, r_s, _ = ref.delta_fwd(*[f64(t) for t in args(x)], 0.4, f64(x["s0"]))
    near(out, r_out[:, :, 0], "out")
    near(state, r_s, "state")


def norm(x, kind, eps=1e-5):
    kw = dict(norm=kind, eps=eps)
    a = (x["xq"], x["xk"], x["wq"], x["wk"])
    q, k = cp.causal_product_qk_rope(*a, x["cos"], x["sin"], **kw)
    dxq, dxk, dwq, dwk = cp.causal_product_qk_rope_bwd(*a, x["gq"], x["gk"], x["cos"], x["sin"], **kw)
    B, _, N, _ = x["xq"].shape
    cos, sin = (np.broadcast_to(f64(t), (B, N, t.shape[-1])) for t in (x["cos"], x["sin"]))
    for xx, w, gy, y, dx, dw in ((x["xq"], x["wq"], x["gq"], q, dxq, dwq),
                                 (x["xk"], x["wk"], x["gk"], k, dxk, dwk)):
        r_dx, r_dw = ref.qk_rope_bwd(f64(xx), f64(w), cos, sin, kind, eps, f64(gy))
        near(y, ref.qk_rope_fwd(f64(xx), f64(w), cos, sin, kind, eps), "y")
        near(dx, r_dx, "dx")
        if dw.dtype == torch.float32:
            near(dw, r_dw, "dw")
        else:  # few elements: each within a step of its type
            step = 2.0 ** (-7 if dw.dtype == torch.bfloat16 else -10)
            assert (np.abs(f64(dw) - r_dw) <= step * np.abs(r_dw) + 1e-6 * np.abs(r_dw).max()).all()


@pytest.mark.parametrize("kind", ["rms", "l2"])
@pytest.mark.parametrize("shape", [(2, 4, 2, 300, 64, 32, "bf16"), (2, 4, 2, 300, 64, 64, "f16"),
                                   (1, 3, 1, 200, 40, 40, "bf16"), (1, 2, 2, 200, 72, 14, "f16"),
                                   (1, 2, 1, 200, 128, 64, "f32"), (1, 2, 1, 150, 248, 130, "f32")],
                         ids=lambda s: "x".join(map(str, s)))
def test_norm(shape, kind):
    *dims, dt = shape
    norm(rope.make(*dims, dt, seed=sum(dims)), kind)


# where R or D is not a multiple of 16 a CTA's first turn is 64 rows (D = 40) or 16
# (D = 248) forward, half backward, on 152 SMs
@pytest.mark.parametrize("shape", [
    (3, 9, 5, 1501, 40, 40, "bf16", False), (3, 9, 5, 1501, 40, 40, "f16", True),
    (2, 5, 3, 1700, 248, 130, "bf16", False), (1, 7, 4, 3001, 72, 14, "f32", True)],
    ids=lambda s: "x".join(map(str, s)))
def test_several_turns_where_rows_turn_by_shuffles(shape):
    *dims, dt, shared = shape
    rope.check(rope.make(*dims, dt, seed=sum(dims), shared=shared), "rms")
