"""The 64-bit references of linear attention with a decay for each head and of
the layer norm against central differences of their own forward, and against
hand examples (CPU)."""
import numpy as np
import pytest

import decay_reference as ref


def _inputs(rng, B=2, H=4, Hk=2, N=6, D=3, M=2):
    return [rng.standard_normal((B, Hk, N, D)), rng.standard_normal((B, Hk, N, D)),
            rng.standard_normal((B, H, N, M)), rng.standard_normal((B, H, D, M))]


def test_hand_example():
    """Half of the state is left at each token."""
    k = np.array([[[[1.0, 0.0], [2.0, 1.0]]]])
    v = np.array([[[[3.0], [5.0]]]])
    out, s, _ = ref.decay_fwd(k, k, v, np.log([0.5]), 2.0, np.array([[[[4.0], [8.0]]]]))
    # S_1 = (2 + 3, 4), S_2 = (2.5 + 10, 2 + 5)
    assert np.allclose(out[0, 0, :, 0], [2 * 5.0, 2 * (2 * 12.5 + 7.0)])
    assert np.allclose(s[0, 0, :, 0], [12.5, 7.0])


def test_lengths_are_shorter_sequences():
    rng = np.random.default_rng(3)
    q, k, v, s0 = _inputs(rng)
    g = -rng.random(4)
    go, gs = rng.standard_normal(v.shape), rng.standard_normal(s0.shape)
    n = [6, 4]
    out, s, _ = ref.decay_fwd(q, k, v, g, 0.7, s0, n)
    d = ref.decay_bwd(q, k, v, g, 0.7, go, gs, s0, n)
    for b in range(2):
        cut = lambda x: x[b:b + 1, :, :n[b]]  # noqa: E731,B023
        o1, s1, _ = ref.decay_fwd(cut(q), cut(k), cut(v), g, 0.7, s0[b:b + 1])
        d1 = ref.decay_bwd(cut(q), cut(k), cut(v), g, 0.7, cut(go), gs[b:b + 1], s0[b:b + 1])
        assert np.array_equal(cut(out), o1) and np.array_equal(s[b], s1[0])
        for x, y in zip(d[:3], d1):
            assert np.array_equal(cut(x), y) and not x[b, :, n[b]:].any()
        assert np.array_equal(d[3][b], d1[3][0])


def test_gradient_against_differences():
    rng = np.random.default_rng(1)
    x = _inputs(rng)
    g = -rng.random(4)
    go, gs = rng.standard_normal(x[2].shape), rng.standard_normal(x[3].shape)

    def loss(a):
        out, s, _ = ref.decay_fwd(*a[:3], g, 0.7, a[3])
        return np.sum(go * out) + np.sum(gs * s)

    d = ref.decay_bwd(*x[:3], g, 0.7, go, gs, x[3])
    for n, (a, grad) in enumerate(zip(x, d)):
        for i in rng.choice(a.size, 10, replace=False):
            y = [t.copy() for t in x]
            h = 1e-5
            y[n].flat[i] += h
            up = loss(y)
            y[n].flat[i] -= 2 * h
            # central differences in 64 bits: h^2 and rounding / h, both ~1e-10
            assert grad.flat[i] == pytest.approx((up - loss(y)) / (2 * h), rel=1e-6, abs=1e-7)


def test_layer_norm_hand_example():
    y = ref.layer_norm_fwd(np.array([[1.0, 3.0]]), np.array([2.0, 10.0]), np.array([0.5, 0.0]), 0.0)
    assert np.allclose(y, [[-2.0 + 0.5, 10.0]])


def test_layer_norm_gradient_against_differences():
    rng = np.random.default_rng(2)
    x, w, b = rng.standard_normal((5, 7)), rng.standard_normal(7), rng.standard_normal(7)
    gy = rng.standard_normal(x.shape)
    loss = lambda *a: np.sum(gy * ref.layer_norm_fwd(*a, 1e-3))  # noqa: E731
    dx, dw, db = ref.layer_norm_bwd(x, w, 1e-3, gy)
    h = 1e-5
    for n, grad in enumerate((dx, dw.sum(0), db.sum(0))):
        for i in rng.choice(grad.size, 7, replace=False):
            a = [t.copy() for t in (x, w, b)]
            a[n].flat[i] += h
            up = loss(*a)
            a[n].flat[i] -= 2 * h
            assert grad.flat[i] == pytest.approx((up - loss(*a)) / (2 * h), rel=1e-6, abs=1e-7)
