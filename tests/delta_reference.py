"""The gated delta rule and the q/k norm with rotation in 64 bits on the CPU,
written from their definitions: token by token, one head at a time, with the
gradients of the recurrence run backwards."""
import numpy as np


def delta_fwd(q, k, v, g, beta, scale, s0=None):
    """(out, S_N, states): states[t] is the state before token t (float64)."""
    B, H, N, M = v.shape
    group, D = H // q.shape[1], q.shape[3]
    out = np.zeros((B, H, N, M))
    states = np.zeros((N + 1, B, H, D, M))
    if s0 is not None:
        states[0] = s0
    for b in range(B):
        for h in range(H):
            for t in range(N):
                kt, qt = k[b, h // group, t], q[b, h // group, t]
                held = np.exp(g[b, h, t]) * states[t, b, h]
                u = beta[b, h, t] * (v[b, h, t] - held.T @ kt)
                states[t + 1, b, h] = held + np.outer(kt, u)
                out[b, h, t] = scale * states[t + 1, b, h].T @ qt
    return out, states[N], states


def delta_bwd(q, k, v, g, beta, scale, go, gs=None, s0=None):
    """(dq, dk, dv, dg, dbeta, dS_0) of <go, out> + <gs, S_N>."""
    _, _, states = delta_fwd(q, k, v, g, beta, scale, s0)
    B, H, N, M = v.shape
    group = H // q.shape[1]
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dg, db, ds0 = np.zeros_like(g), np.zeros_like(beta), np.zeros_like(states[0])
    for b in range(B):
        for h in range(H):
            hk = h // group
            ds = np.zeros_like(states[0, b, h]) if gs is None else gs[b, h].copy()
            for t in reversed(range(N)):
                kt, qt, a = k[b, hk, t], q[b, hk, t], np.exp(g[b, h, t])
                held = a * states[t, b, h]
                miss = v[b, h, t] - held.T @ kt
                dq[b, hk, t] += scale * states[t + 1, b, h] @ go[b, h, t]
                ds = ds + scale * np.outer(qt, go[b, h, t])
                du = ds.T @ kt
                dk[b, hk, t] += ds @ (beta[b, h, t] * miss)
                db[b, h, t] = du @ miss
                dv[b, h, t] = beta[b, h, t] * du
                dk[b, hk, t] -= held @ dv[b, h, t]
                ds = ds - np.outer(kt, dv[b, h, t])
                dg[b, h, t] = np.sum(ds * held)
                ds = a * ds
            ds0[b, h] = ds
    return dq, dk, dv, dg, db, ds0


def qk_rope_fwd(x, w, cos, sin, norm, eps):
    """x [B,H,N,D], w [D] or None, cos and sin [B,N,R/2]."""
    D = x.shape[-1]
    ss = np.sum(x * x, -1, keepdims=True) / (D if norm == "rms" else 1)
    y = x / np.sqrt(ss + eps) * (1.0 if w is None else w)
    half = cos.shape[-1]
    out = y.copy()
    for i in range(half):
        c, s = cos[:, None, :, i], sin[:, None, :, i]
        out[..., i] = y[..., i] * c - y[..., half + i] * s
        out[..., half + i] = y[..., half + i] * c + y[..., i] * s
    return out


def qk_rope_bwd(x, w, cos, sin, norm, eps, gy):
    """(dx, dw) of <gy, y>."""
    D = x.shape[-1]
    c = 1.0 / D if norm == "rms" else 1.0
    r = 1.0 / np.sqrt(c * np.sum(x * x, -1, keepdims=True) + eps)
    half = cos.shape[-1]
    d = gy.copy()
    for i in range(half):
        co, s = cos[:, None, :, i], sin[:, None, :, i]
        d[..., i] = gy[..., i] * co + gy[..., half + i] * s
        d[..., half + i] = gy[..., half + i] * co - gy[..., i] * s
    t = d * (1.0 if w is None else w)
    dx = r * (t - c * r * r * x * np.sum(x * t, -1, keepdims=True))
    return dx, np.sum(d * x * r, (0, 1, 2))
