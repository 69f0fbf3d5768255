"""The gated delta rule and the q/k norm on the GPU (``-m gpu``) at the sizes
that choose between their kernels' blocks: value columns to a CTA by the number
of heads, blocks that end inside the matrix, lanes that hold part of a row.
Bounds and references are those of the operators' other tests."""
import pytest
import torch

import test_delta_gpu as delta
import test_qk_rope_gpu as rope

pytestmark = pytest.mark.gpu


# B, H, Hk, N, D, M, dtype, carried state: 64, 32 and 16 columns to a CTA, with
# and without a last block cut short
@pytest.mark.parametrize("shape", [
    (2, 40, 20, 70, 64, 72, "f32", True), (2, 80, 80, 33, 24, 40, "f32", False),
    (2, 32, 32, 45, 64, 64, "f16", True), (1, 60, 60, 34, 136, 40, "bf16", True),
    (1, 20, 10, 66, 200, 24, "f32", False), (1, 1, 1, 95, 31, 17, "f32", True),
    (2, 80, 40, 65, 64, 64, "bf16", True), (1, 12, 12, 129, 104, 40, "bf16", True)],
    ids=lambda s: "x".join(map(str, s)))
def test_blocks(shape):
    B, H, Hk, N, D, M, dt, carry = shape
    delta.check(delta.make(B, H, Hk, N, D, M, delta.DT[dt], seed=B + H + N + D, carry=carry))


# norms of rows of one, three, seven and sixteen lanes' worth, heads that do not
# divide a warp's rows
@pytest.mark.parametrize("shape", [
    (2, 3, 1, 41, 16, 16, "bf16"), (1, 5, 2, 77, 48, 0, "f16"), (2, 3, 3, 130, 112, 96, "bf16"),
    (1, 7, 1, 300, 256, 128, "bf16"), (1, 2, 2, 50, 32, 16, "f32"), (3, 6, 2, 19, 160, 160, "f16")],
    ids=lambda s: "x".join(map(str, s)))
def test_rows(shape):
    *dims, dt = shape
    rope.check(rope.make(*dims, dt, seed=sum(dims)), "rms")


def test_heads_past_a_turn_of_the_blocks():
    """More rows than one turn of every CTA: the walk's places over tokens and
    batches, with one table of angles a batch."""
    rope.check(rope.make(3, 5, 2, 1500, 64, 32, "bf16", seed=3), "l2")


@pytest.mark.parametrize("dt,D,M", [("bf16", 64, 40), ("f32", 48, 33), ("f16", 128, 104),
                                    ("bf16", 256, 72), ("f32", 7, 5)])
def test_one_token(dt, D, M):
    """One token after the first 20 is the 21st row of a forward."""
    x = delta.make(3, 4, 2, 21, D, M, delta.DT[dt], seed=D + M, carry=True)
    r_out, r_s, _ = delta.ref.delta_fwd(*[delta.f64(t) for t in delta.args(x)], 0.3,
                                        delta.f64(x["s0"]))
    cut = [t[:, :, :20].contiguous() for t in delta.args(x)]
    last = [t[:, :, 20].contiguous() for t in delta.args(x)]
    _, s = delta.cp.causal_product_fwd_delta(*cut, state_in=x["s0"], return_state=True, scale=0.3)
    out = delta.cp.causal_product_decode_delta(*last, s, scale=0.3)
    torch.cuda.synchronize()
    delta.close(out, r_out[:, :, 20], "out")
    delta.close(s, r_s, "state")
