"""The 64-bit references of the gated delta rule and of the q/k norm with
rotation against central differences of their own forward, and against hand
examples (CPU)."""
import numpy as np
import pytest

import delta_reference as ref


def _delta_inputs(rng, B=1, H=4, Hk=2, N=7, D=3, M=2):
    q, k = rng.standard_normal((B, Hk, N, D)), rng.standard_normal((B, Hk, N, D))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    return [q, k, rng.standard_normal((B, H, N, M)), -rng.random((B, H, N)), rng.random((B, H, N)),
            rng.standard_normal((B, H, D, M))]


def test_delta_hand_example():
    """Two tokens with the same unit key: the second write replaces the first."""
    k = np.array([[[[1.0, 0.0], [1.0, 0.0]]]])
    v = np.array([[[[3.0], [5.0]]]])
    out, s, _ = ref.delta_fwd(k, k, v, np.zeros((1, 1, 2)), np.ones((1, 1, 2)), 1.0)
    assert np.array_equal(out[0, 0, :, 0], [3.0, 5.0])
    assert np.array_equal(s[0, 0, :, 0], [5.0, 0.0])
    # half strength and half decay: 1.5, then 0.75 + 0.5 (5 - 0.75)
    out, _, _ = ref.delta_fwd(k, k, v, np.full((1, 1, 2), np.log(0.5)), np.full((1, 1, 2), 0.5), 2.0)
    assert np.allclose(out[0, 0, :, 0], [2 * 1.5, 2 * 2.875])


def test_delta_gradient_against_differences():
    rng = np.random.default_rng(1)
    x = _delta_inputs(rng)
    go, gs = rng.standard_normal(x[2].shape), rng.standard_normal(x[5].shape)

    def loss(a):
        out, s, _ = ref.delta_fwd(*a[:5], 0.7, a[5])
        return np.sum(go * out) + np.sum(gs * s)

    d = ref.delta_bwd(*x[:5], 0.7, go, gs, x[5])
    for n, (a, grad) in enumerate(zip(x, d)):
        for i in rng.choice(a.size, 10, replace=False):
            y = [t.copy() for t in x]
            h = 1e-5
            y[n].flat[i] += h
            up = loss(y)
            y[n].flat[i] -= 2 * h
            # central differences in 64 bits: h^2 and rounding / h, both ~1e-10
            assert grad.flat[i] == pytest.approx((up - loss(y)) / (2 * h), rel=1e-6, abs=1e-7)


@pytest.mark.parametrize("norm", ["rms", "l2"])
def test_rope_gradient_against_differences(norm):
    rng = np.random.default_rng(2)
    x, w = rng.standard_normal((2, 2, 3, 8)), rng.standard_normal(8)
    ang = rng.standard_normal((2, 3, 3))
    gy = rng.standard_normal(x.shape)
    loss = lambda a, b: np.sum(gy * ref.qk_rope_fwd(a, b, np.cos(ang), np.sin(ang), norm, 1e-3))  # noqa: E731
    dx, dw = ref.qk_rope_bwd(x, w, np.cos(ang), np.sin(ang), norm, 1e-3, gy)
    h = 1e-5
    for i in rng.choice(x.size, 12, replace=False):
        e = np.zeros_like(x)
        e.flat[i] = h
        assert dx.flat[i] == pytest.approx((loss(x + e, w) - loss(x - e, w)) / (2 * h), rel=1e-6, abs=1e-7)
    for i in range(8):
        e = np.zeros_like(w)
        e[i] = h
        assert dw[i] == pytest.approx((loss(x, w + e) - loss(x, w - e)) / (2 * h), rel=1e-6, abs=1e-7)


def test_rope_keeps_the_norm():
    rng = np.random.default_rng(3)
    x, ang = rng.standard_normal((1, 1, 4, 16)), rng.standard_normal((1, 4, 5))
    y = ref.qk_rope_fwd(x, None, np.cos(ang), np.sin(ang), "l2", 0.0)
    assert np.allclose(np.linalg.norm(y, axis=-1), 1.0)
    assert np.allclose(y[..., 10:], x[..., 10:] / np.linalg.norm(x, axis=-1, keepdims=True))
