"""Host-side checks of the gated delta rule's and the q/k norm's C entry points:
sizes, and refusals that come before any CUDA work (no GPU needed; the
pointers are never followed)."""
import ctypes

import pytest
import torch

import prefix_sum_outer_gb300 as cp

F32, BF16, F16 = 0, 1, 2
(OK, INVALID_ARG, UNSUPPORTED_SHAPE, UNSUPPORTED_DTYPE, MISALIGNED, WS_TOO_SMALL) = range(6)
GAP = 1 << 32  # between the made-up buffers


@pytest.fixture(scope="module")
def lib():
    return cp.load_library()


def buffers(n):
    return [GAP * (i + 1) for i in range(n)]


def fwd(lib, q=None, B=1, H=2, Hk=2, N=8, D=16, M=16, dtype=BF16, scale=1.0, ws=0, ws_n=0,
        ckpt=0, ckpt_n=0, **put):
    names = ("q", "k", "v", "g", "beta", "out", "state_in", "state_out")
    p = dict(zip(names, buffers(8)))
    if q is not None:
        p["q"] = q
    p.update(put)
    return lib.causal_product_fwd_delta(*(p[n] for n in names), ckpt, ckpt_n, scale, B, H, Hk, N,
                                        D, M, dtype, ws, ws_n, 0)


def bwd(lib, B=1, H=2, Hk=2, N=8, D=16, M=16, dtype=BF16, scale=1.0, ws=0, ws_n=0,
        ckpt_n=1 << 20, **put):
    names = ("q", "k", "v", "g", "beta", "grad_out", "ckpt")
    outs = ("gs_out", "dq", "dk", "dv", "dg", "db", "gs_in")
    p = dict(zip(names + outs, buffers(14)))
    p.update(put)
    return lib.causal_product_bwd_delta(*(p[n] for n in names), ckpt_n, *(p[n] for n in outs),
                                        scale, B, H, Hk, N, D, M, dtype, ws, ws_n, 0)


def decode(lib, B=2, H=2, Hk=2, D=16, M=16, dtype=BF16, scale=1.0, pool=4, **put):
    names = ("q", "k", "v", "g", "beta", "out", "state", "slots")
    p = dict(zip(names, buffers(8)))
    p.update(put)
    return lib.causal_product_decode_delta(*(p[n] for n in names), pool, scale, B, H, Hk, D, M,
                                           dtype, 0)


SHAPES = [
    (dict(H=3, Hk=2), INVALID_ARG),          # heads that no key head serves
    (dict(H=1, Hk=2), INVALID_ARG),
    (dict(Hk=0), INVALID_ARG),
    (dict(B=0), INVALID_ARG),
    (dict(scale=float("nan")), INVALID_ARG),
    (dict(scale=float("inf")), INVALID_ARG),
    (dict(D=264), UNSUPPORTED_SHAPE),
    (dict(M=257, dtype=F32), UNSUPPORTED_SHAPE),
    (dict(D=0), UNSUPPORTED_SHAPE),
    (dict(D=12), UNSUPPORTED_SHAPE),         # bf16: multiples of 8
    (dict(M=4), UNSUPPORTED_SHAPE),
    (dict(dtype=7), UNSUPPORTED_DTYPE),
    (dict(q=0), INVALID_ARG),
    (dict(out=0), INVALID_ARG),
    (dict(beta=0), INVALID_ARG),
    (dict(q=GAP + 8), MISALIGNED),
    (dict(g=4 * GAP + 2), MISALIGNED),
    (dict(out=6 * GAP + 4), MISALIGNED),
    (dict(out=3 * GAP), INVALID_ARG),        # out on v
]


@pytest.mark.parametrize("put,want", SHAPES)
def test_forward_refusals(lib, put, want):
    assert fwd(lib, **put) == want


@pytest.mark.parametrize("put,want", [(p, w) for p, w in SHAPES if "out" not in p])
def test_backward_refusals(lib, put, want):
    assert bwd(lib, **put) == want


@pytest.mark.parametrize("put,want", SHAPES)
def test_decode_refusals(lib, put, want):
    assert decode(lib, **put) == want


def test_negative_rows(lib):
    assert fwd(lib, N=-1) == INVALID_ARG
    assert bwd(lib, N=-1) == INVALID_ARG


def test_states_and_checkpoints(lib):
    assert fwd(lib, state_in=7 * GAP + 4) == MISALIGNED
    assert fwd(lib, state_out=7 * GAP) == INVALID_ARG          # the state it starts from
    n = lib.causal_product_delta_checkpoint_size(1, 2, 2, 8, 16, 16, BF16)
    assert n > 0
    assert fwd(lib, ckpt=20 * GAP, ckpt_n=n - 1) == WS_TOO_SMALL
    assert bwd(lib, ckpt_n=n - 1) == WS_TOO_SMALL
    assert bwd(lib, ckpt=0) == INVALID_ARG
    assert bwd(lib, dq=GAP) == INVALID_ARG                      # on q
    assert bwd(lib, dk=9 * GAP) == INVALID_ARG                  # on dq
    assert bwd(lib, dg=12 * GAP + 2) == MISALIGNED


def test_workspaces(lib):
    for back, call in ((0, fwd), (1, bwd)):
        n = lib.causal_product_delta_workspace_size(1, 2, 2, 8, 16, 16, BF16, back)
        assert n > 0
        assert call(lib, ws=30 * GAP, ws_n=n - 1) == WS_TOO_SMALL
    # parameters the calls refuse have no size
    for bad in ((1, 3, 2, 8, 16, 16, BF16), (1, 2, 2, 8, 300, 16, F32), (1, 2, 2, -1, 16, 16, F32)):
        assert lib.causal_product_delta_workspace_size(*bad, 0) == 0
        assert lib.causal_product_delta_checkpoint_size(*bad) == 0


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("D,M", [(64, 64), (128, 200), (256, 256)])
def test_checkpoints_grow_with_the_rows(lib, dtype, D, M):
    """A checkpoint holds at least one state per chunk of rows, a size that 32
    bits do not hold for long sequences of many heads."""
    last = -1
    for N in (0, 1, 32, 64, 65, 4096):
        n = lib.causal_product_delta_checkpoint_size(2, 4, 2, N, D, M, dtype)
        assert n >= last
        last = n
    assert last >= 2 * 4 * (4096 // 64) * D * M * 2
    big = lib.causal_product_delta_checkpoint_size(512, 16, 16, 1 << 16, D, M, dtype)
    assert big > 1 << 32


def test_pool_of_states(lib):
    assert decode(lib, pool=0) == INVALID_ARG
    assert decode(lib, pool=1, slots=0) == INVALID_ARG         # fewer states than sequences
    assert decode(lib, slots=8 * GAP + 2) == MISALIGNED
    assert decode(lib, state=6 * GAP) == INVALID_ARG           # on out
    assert decode(lib, slots=7 * GAP) == INVALID_ARG           # inside the states


def rope(lib, back=False, B=1, Hq=2, Hk=1, N=8, D=16, R=16, dtype=BF16, norm=0, eps=1e-6,
         sq=(256, 128, 16), sk=(128, 128, 16), cs_batch=0, ws=0, ws_n=0, **put):
    names = ("xq", "xk", "wq", "wk", "cos", "sin", "a", "b", "dxq", "dxk", "dwq", "dwk")
    p = dict(zip(names, buffers(12)))
    p.update(put)
    st = [None if s is None else (ctypes.c_int64 * 3)(*s) for s in (sq, sk)]
    head = (p["xq"], st[0], p["xk"], st[1], p["wq"], p["wk"], p["cos"], p["sin"], cs_batch,
            p["a"], p["b"])
    tail = (norm, eps, B, Hq, Hk, N, D, R, dtype)
    if not back:
        return lib.causal_product_qk_rope(*head, *tail, 0)
    return lib.causal_product_qk_rope_bwd(*head, p["dxq"], p["dxk"], p["dwq"], p["dwk"], *tail,
                                          ws, ws_n, 0)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("put,want", [
    (dict(B=0), INVALID_ARG),
    (dict(N=-1), INVALID_ARG),
    (dict(norm=2), INVALID_ARG),
    (dict(eps=-1.0), INVALID_ARG),
    (dict(eps=float("nan")), INVALID_ARG),
    (dict(D=12), UNSUPPORTED_SHAPE),
    (dict(D=264), UNSUPPORTED_SHAPE),
    (dict(R=18), UNSUPPORTED_SHAPE),         # more features than the row has
    (dict(R=7), UNSUPPORTED_SHAPE),
    (dict(N=1 << 31), UNSUPPORTED_SHAPE),    # rows past 32 bits
    (dict(dtype=9), UNSUPPORTED_DTYPE),
    (dict(sq=None), INVALID_ARG),
    (dict(sk=(128, -16, 16)), INVALID_ARG),
    (dict(xq=0), INVALID_ARG),
    (dict(cos=0), INVALID_ARG),
    (dict(cs_batch=-1), INVALID_ARG),
    (dict(xk=2 * GAP + 1), MISALIGNED),
    (dict(a=7 * GAP + 8), MISALIGNED),
    (dict(sin=6 * GAP + 2), MISALIGNED),
])
def test_rope_refusals(lib, put, want, back):
    assert rope(lib, back, **put) == want


def test_rope_overlaps_and_workspace(lib):
    assert rope(lib, a=GAP) == INVALID_ARG                     # q on xq
    assert rope(lib, b=7 * GAP) == INVALID_ARG                 # k on q
    assert rope(lib, True, dxq=7 * GAP) == INVALID_ARG         # on grad_q
    assert rope(lib, True, dwq=0) == INVALID_ARG               # a weight without its gradient
    assert rope(lib, True, wk=0) == INVALID_ARG                # and the other way round
    n = lib.causal_product_qk_rope_workspace_size(1, 2, 1, 8, 16, BF16)
    assert n > 0
    assert rope(lib, True, ws=30 * GAP, ws_n=n - 1) == WS_TOO_SMALL
    assert lib.causal_product_qk_rope_workspace_size(1, 2, 1, 8, 12, BF16) == 0


def test_python_calls_refuse_cpu_tensors():
    q = torch.zeros(1, 2, 4, 16)
    g = torch.zeros(1, 2, 4)
    with pytest.raises(RuntimeError):
        cp.causal_product_fwd_delta(q, q, q, g, g)
    with pytest.raises(RuntimeError):
        cp.causal_product_decode_delta(q[:, :, 0], q[:, :, 0], q[:, :, 0], g[:, :, 0], g[:, :, 0],
                                       torch.zeros(1, 2, 16, 16))
    with pytest.raises(RuntimeError):
        cp.causal_product_qk_rope(q, q)
