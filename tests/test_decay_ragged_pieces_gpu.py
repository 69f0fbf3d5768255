"""Linear attention with a decay for each head where a sequence is cut into pieces
and a batch is ragged at once (``-m gpu``): sequences that end in early pieces, at
the end of a piece or a part of one, a row before and a row behind it, with nothing
at all, and padding full of NaN.  All six results against 64 bits.

Few heads over 11 to 21 tiles of 128 rows are cut into pieces of one to a few
tiles, differently for the forward, the backward's products in one launch and
their own; every tile's end is a length here, so every piece's end and every
part's is.

The reference takes each sequence alone, in blocks of 50 rows, from the
recurrence's sums in 64 bits.  Bounds: a result in bf16 is at most 2^-8 of its
size off in each sequence, and 2e-4 from the 64-bit one rounded to bf16 over the
batch (test_decay_precision_gpu.py); one in fp32 2e-6 (test_decay_gpu.py)."""
import pytest
import torch

from test_decay_gpu import DT, NAMES, TOL, make, results

pytestmark = pytest.mark.gpu

BLOCK = 50


def walk(a, b, c, g, s):
    """sum_{j<=i} e^{g(i-j)} (a_i . b_j) c_j + e^{g(i+1)} s^T a_i for rows [H,n,.], and
    the state behind the last row."""
    out = []
    for i in range(0, a.shape[1], BLOCK):
        x, y, z = (t[:, i:i + BLOCK] for t in (a, b, c))
        r = torch.arange(x.shape[1], device=a.device, dtype=torch.float64)
        gap = r[:, None] - r
        w = torch.where(gap >= 0, torch.exp(g[:, None, None] * gap.clamp_min(0)), 0.0)
        up, down = torch.exp(g[:, None] * (r + 1)), torch.exp(g[:, None] * (len(r) - 1 - r))
        out.append((w * (x @ y.mT)) @ z + up[..., None] * (x @ s))
        s = torch.exp(g * len(r))[:, None, None] * s + (down[..., None] * y).mT @ z
    return (torch.cat(out, 1) if out else c[:, :0]), s


def wanted(x, b, n, scale=0.3):
    """The six results of sequence b's first n rows."""
    d = lambda t: x[t][b].double()  # noqa: E731
    H, Hk = x["v"].shape[1], x["q"].shape[1]
    q, k = (d(t)[:, :n].repeat_interleave(H // Hk, 0) for t in ("q", "k"))
    v, go, g = d("v")[:, :n], scale * d("go")[:, :n], x["g"].double()
    out, end = walk(q, k, v, g, d("s0"))
    # backwards: the gradient of the state behind the last row, one step nearer
    gs = d("gs") / torch.exp(g)[:, None, None]
    flip = lambda t: t.flip(1)  # noqa: E731
    dq, _ = walk(go, v, k, g, d("s0").mT)
    dv, ds = walk(flip(k), flip(q), flip(go), g, gs)
    dk, _ = walk(flip(v), flip(go), flip(q), g, gs.mT)
    few = lambda t: t.unflatten(0, (Hk, H // Hk)).sum(1)  # noqa: E731
    return dict(zip(NAMES, (scale * out, end, few(dq), few(flip(dk)), flip(dv),
                            ds * torch.exp(g)[:, None, None])))


def norm(t):
    return float(t.norm())


def check(shape, lengths, seed):
    B, H, Hk, N, D, M = shape
    x = make(*shape, DT["bf16"], seed=seed, carry=True, lengths=lengths,
             rates=[-0.002 * 6.0 ** i for i in range(H)])
    clean = dict(x)
    for t in ("q", "k", "v", "go"):
        x[t] = x[t].clone()
        for b, n in enumerate(lengths):
            x[t][b, :, n:] = float("nan")
            x[t][b, :, n + 1::3] = float("inf")
    got = results(x)
    off, size = dict.fromkeys(NAMES, 0.0), dict.fromkeys(NAMES, 0.0)
    for b, n in enumerate(lengths):
        want = wanted(clean, b, n)
        for name in NAMES:
            a, w = got[name][b], want[name]
            if name in ("out", "dq", "dk", "dv"):
                assert not a[:, n:].any(), (name, n)
                a = a[:, :n]
            assert norm(a.double() - w) <= TOL[a.dtype] * norm(w), (name, n)
            off[name] += norm(a.double() - w.to(a.dtype).double()) ** 2
            size[name] += norm(w) ** 2
        if n == 0:
            assert torch.equal(got["state"][b], x["s0"][b])
            assert torch.equal(got["dstate"][b], x["gs"][b])
    for name in NAMES:
        if got[name].dtype == torch.bfloat16:
            assert off[name] <= 2e-4 ** 2 * size[name], name


# B, H, Hk, N, D, M: pieces of one tile, of two, of six that are summed in parts
SHAPES = [(6, 2, 1, 1500, 64, 64), (6, 2, 2, 2700, 128, 128), (6, 2, 1, 2700, 40, 72),
          (6, 3, 3, 1900, 64, 128), (6, 6, 3, 2700, 64, 64)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_every_end(shape):
    B, N = shape[0], shape[3]
    ends = [0, 1, N, N - 1] + [128 * t + d for t in range(1, N // 128 + 1) for d in (-1, 0, 1)]
    ends = [n for n in ends if n <= N]
    # far ends side by side
    step = -(-len(ends) // B)
    for i in range(step):
        lengths = [ends[(i + j * step) % len(ends)] for j in range(B)]
        check(shape, lengths, seed=100 + i)
