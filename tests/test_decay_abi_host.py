"""Host-side checks of the C entry points of linear attention with a decay for
each head and of the layer norm: sizes, and refusals that come before any CUDA
work (no GPU needed; the pointers are never followed)."""
import ctypes

import pytest
import torch

import prefix_sum_outer_gb300 as cp

F32, BF16, F16 = 0, 1, 2
(OK, INVALID_ARG, UNSUPPORTED_SHAPE, UNSUPPORTED_DTYPE, MISALIGNED, WS_TOO_SMALL) = range(6)
GAP = 1 << 40  # between the made-up buffers


@pytest.fixture(scope="module")
def lib():
    return cp.load_library()


def buffers(names, put):
    p = {n: GAP * (i + 1) for i, n in enumerate(names)}
    assert set(put) <= set(p)
    p.update(put)
    return p


def fwd(lib, B=1, H=2, Hk=2, N=8, D=16, M=16, dtype=BF16, scale=1.0, ws=0, ws_n=0, **put):
    names = ("q", "k", "v", "g", "out", "state_in", "state_out", "lengths")
    p = buffers(names, put)
    return lib.causal_product_fwd_decay(*(p[n] for n in names), scale, B, H, Hk, N, D, M, dtype,
                                        ws, ws_n, 0)


def bwd(lib, B=1, H=2, Hk=2, N=8, D=16, M=16, dtype=BF16, scale=1.0, ws=0, ws_n=0, **put):
    names = ("q", "k", "v", "g", "go", "state_in", "gs_out", "dq", "dk", "dv", "gs_in", "lengths")
    p = buffers(names, put)
    return lib.causal_product_bwd_decay(*(p[n] for n in names), scale, B, H, Hk, N, D, M, dtype,
                                        ws, ws_n, 0)


def decode(lib, B=2, H=2, Hk=2, D=16, M=16, dtype=BF16, scale=1.0, pool=4, **put):
    names = ("q", "k", "v", "g", "out", "state", "slots")
    p = buffers(names, put)
    return lib.causal_product_decode_decay(*(p[n] for n in names), pool, scale, B, H, Hk, D, M,
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
    (dict(g=0), INVALID_ARG),
    (dict(q=GAP + 8), MISALIGNED),
    (dict(g=4 * GAP + 2), MISALIGNED),
]


@pytest.mark.parametrize("put,want", SHAPES + [
    (dict(out=0), INVALID_ARG), (dict(out=6 * GAP + 4), MISALIGNED),
    (dict(out=3 * GAP), INVALID_ARG),                               # out on v
    (dict(N=-1), INVALID_ARG), (dict(N=1 << 31), UNSUPPORTED_SHAPE),
    (dict(state_in=6 * GAP + 4), MISALIGNED),
    (dict(state_out=6 * GAP), INVALID_ARG),                         # the state it starts from
    (dict(lengths=8 * GAP + 2), MISALIGNED), (dict(out=8 * GAP), INVALID_ARG)])
def test_forward_refusals(lib, put, want):
    assert fwd(lib, **put) == want


@pytest.mark.parametrize("put,want", SHAPES + [
    (dict(go=0), INVALID_ARG), (dict(dq=0), INVALID_ARG), (dict(dv=0), INVALID_ARG),
    (dict(dq=GAP), INVALID_ARG), (dict(dk=8 * GAP), INVALID_ARG),   # on q, on dq
    (dict(gs_in=7 * GAP), INVALID_ARG), (dict(gs_in=11 * GAP + 8), MISALIGNED),
    (dict(N=-1), INVALID_ARG), (dict(lengths=12 * GAP + 1), MISALIGNED)])
def test_backward_refusals(lib, put, want):
    assert bwd(lib, **put) == want


@pytest.mark.parametrize("put,want", SHAPES + [
    (dict(out=0), INVALID_ARG), (dict(state=0), INVALID_ARG), (dict(pool=0), INVALID_ARG),
    (dict(pool=1, slots=0), INVALID_ARG), (dict(out=3 * GAP), INVALID_ARG),
    (dict(state=GAP), INVALID_ARG), (dict(slots=7 * GAP + 2), MISALIGNED)])
def test_decode_refusals(lib, put, want):
    assert decode(lib, **put) == want


def test_workspaces(lib):
    for back, call in ((0, fwd), (1, bwd)):
        n = lib.causal_product_decay_workspace_size(1, 2, 2, 8, 16, 16, BF16, back)
        assert n > 0
        assert call(lib, ws=30 * GAP, ws_n=n - 1) == WS_TOO_SMALL
    # parameters the calls refuse have no size
    for bad in ((1, 3, 2, 8, 16, 16, BF16), (1, 2, 2, 8, 300, 16, F32), (1, 2, 2, -1, 16, 16, F32)):
        assert lib.causal_product_decay_workspace_size(*bad, 0) == 0


def norm(lib, strides=(512, 256, 32), per_head=0, major=0, eps=1e-5, B=2, H=2, N=8, C=32, dtype=BF16,
         **put):
    names = ("x", "w", "b", "y")
    p = buffers(names, put)
    s = None if strides is None else (ctypes.c_int64 * 3)(*strides)
    return lib.causal_product_layer_norm(p["x"], s, p["w"], p["b"], per_head, p["y"], major, eps,
                                         B, H, N, C, dtype, 0)


def norm_bwd(lib, strides=(512, 256, 32), per_head=0, major=0, eps=1e-5, B=2, H=2, N=8, C=32,
             dtype=BF16, ws=0, ws_n=0, **put):
    names = ("x", "w", "gy", "dx", "dw", "db")
    p = buffers(names, put)
    s = None if strides is None else (ctypes.c_int64 * 3)(*strides)
    return lib.causal_product_layer_norm_bwd(p["x"], s, p["w"], per_head, p["gy"], major, p["dx"],
                                             p["dw"], p["db"], eps, B, H, N, C, dtype, ws, ws_n, 0)


NORMS = [
    (dict(B=0), INVALID_ARG), (dict(H=0), INVALID_ARG), (dict(N=-1), INVALID_ARG),
    (dict(C=0), UNSUPPORTED_SHAPE), (dict(C=32769), UNSUPPORTED_SHAPE),
    (dict(H=65536), UNSUPPORTED_SHAPE), (dict(B=1 << 16, N=1 << 15), UNSUPPORTED_SHAPE),
    (dict(B=1 << 40, N=1 << 40), UNSUPPORTED_SHAPE),
    (dict(dtype=5), UNSUPPORTED_DTYPE), (dict(eps=-1.0), INVALID_ARG),
    (dict(eps=float("nan")), INVALID_ARG), (dict(eps=float("inf")), INVALID_ARG),
    (dict(strides=None), INVALID_ARG), (dict(strides=(1, -1, 1)), INVALID_ARG),
    (dict(x=0), INVALID_ARG), (dict(x=GAP + 1), MISALIGNED),
    (dict(w=2 * GAP + 2, dtype=F32), MISALIGNED),
]


@pytest.mark.parametrize("put,want", NORMS + [
    (dict(y=0), INVALID_ARG), (dict(y=4 * GAP + 8), MISALIGNED), (dict(y=GAP), INVALID_ARG),
    (dict(y=2 * GAP), INVALID_ARG), (dict(b=3 * GAP + 1), MISALIGNED)])
def test_norm_refusals(lib, put, want):
    assert norm(lib, **put) == want


@pytest.mark.parametrize("put,want", NORMS + [
    (dict(gy=0), INVALID_ARG), (dict(dx=0), INVALID_ARG), (dict(gy=3 * GAP + 8), MISALIGNED),
    (dict(dx=3 * GAP), INVALID_ARG), (dict(dw=GAP), INVALID_ARG), (dict(db=5 * GAP), INVALID_ARG),
    (dict(w=0), INVALID_ARG),                                       # dw without w
    (dict(db=6 * GAP + 1), MISALIGNED)])
def test_norm_backward_refusals(lib, put, want):
    assert norm_bwd(lib, **put) == want


def test_norm_workspaces(lib):
    n = lib.causal_product_layer_norm_workspace_size(2, 2, 8, 32, BF16)
    assert n > 0
    assert norm_bwd(lib, ws=30 * GAP, ws_n=n - 1) == WS_TOO_SMALL
    assert norm_bwd(lib, ws=30 * GAP + 16, ws_n=n) == MISALIGNED
    assert lib.causal_product_layer_norm_workspace_size(2, 2, 8, 0, BF16) == 0


def test_python_refusals_without_a_gpu():
    q = torch.zeros(1, 2, 4, 8)
    g = torch.zeros(2)
    with pytest.raises(ValueError):
        cp.causal_product_fwd_decay(q, q[:, :1], q, g)
    with pytest.raises(ValueError):
        cp.causal_product_fwd_decay(q, q, q, torch.zeros(3))
    with pytest.raises(ValueError):
        cp.causal_product_fwd_decay(q, q, q, g.double())
    with pytest.raises(ValueError):
        cp.causal_product_fwd_decay(q, q, q, g, lengths=torch.zeros(1, dtype=torch.int64))
    with pytest.raises(RuntimeError):
        cp.causal_product_fwd_decay(q, q, q, g)
    with pytest.raises(RuntimeError):
        cp.causal_product_fwd_decay(q, q, q, g, lengths=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        cp.causal_product_decay(q, q, q, g.requires_grad_(True))    # the decay is a constant
    with pytest.raises(RuntimeError):
        cp.causal_product_layer_norm(q)
    with pytest.raises(ValueError):
        cp.causal_product_layer_norm(q[0], token_major=True)
    with pytest.raises(ValueError):
        cp.causal_product_layer_norm(torch.zeros(3))
