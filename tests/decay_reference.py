"""Linear attention with a decay for each head, and the layer norm, in 64 bits
on the CPU, written from their definitions: token by token, the gradients of the
recurrence run backwards."""
import numpy as np


def _many(x, H):
    return np.repeat(x, H // x.shape[1], axis=1)


def decay_fwd(q, k, v, g, scale, s0=None, lengths=None):
    """(out, S_n, states): states[t] is the state before token t (float64);
    tokens past a sequence's length leave it and give zero."""
    B, H, N, M = v.shape
    q, k = _many(q, H), _many(k, H)
    n = np.full(B, N) if lengths is None else np.asarray(lengths)
    a = np.exp(g)[None, :, None, None]
    out = np.zeros((B, H, N, M))
    s = np.zeros((B, H, q.shape[3], M)) if s0 is None else s0.copy()
    states = []
    for t in range(N):
        states.append(s)
        on = (t < n)[:, None, None, None]
        kv = np.where(on, k[:, :, t, :, None], 0.0) * np.where(on, v[:, :, t, None, :], 0.0)
        s = np.where(on, a * s + kv, s)
        qt = np.where(on[..., 0], q[:, :, t], 0.0)
        out[:, :, t] = scale * np.einsum("bhdm,bhd->bhm", s, qt)
    return out, s, states


def decay_bwd(q, k, v, g, scale, go, gs=None, s0=None, lengths=None):
    """(dq, dk, dv, dS_0) of <go, out> + <gs, S_n>."""
    B, H, N, M = v.shape
    Hk, D = q.shape[1], q.shape[3]
    _, end, states = decay_fwd(q, k, v, g, scale, s0, lengths)
    states = states + [end]
    q, k = _many(q, H), _many(k, H)
    n = np.full(B, N) if lengths is None else np.asarray(lengths)
    a = np.exp(g)[None, :, None, None]
    dq, dk, dv = np.zeros((B, H, N, D)), np.zeros((B, H, N, D)), np.zeros((B, H, N, M))
    ds = np.zeros((B, H, D, M)) if gs is None else gs.copy()
    for t in reversed(range(N)):
        on = (t < n)[:, None, None]
        qt, kt, vt, gt = (np.where(on, x[:, :, t], 0.0) for x in (q, k, v, go))
        dq[:, :, t] = scale * np.einsum("bhdm,bhm->bhd", states[t + 1], gt)
        ds = ds + scale * qt[..., None] * gt[:, :, None, :]
        dk[:, :, t] = np.where(on, np.einsum("bhdm,bhm->bhd", ds, vt), 0.0)
        dv[:, :, t] = np.where(on, np.einsum("bhdm,bhd->bhm", ds, kt), 0.0)
        ds = np.where(on[..., None], a * ds, ds)
    few = lambda x: x.reshape(B, Hk, H // Hk, N, D).sum(2)  # noqa: E731
    return few(dq), few(dk), dv, ds


def layer_norm_fwd(x, w, b, eps):
    """Rows in the last dimension; w and b broadcast against x."""
    mu = x.mean(-1, keepdims=True)
    xh = (x - mu) / np.sqrt(((x - mu) ** 2).mean(-1, keepdims=True) + eps)
    return xh * (1.0 if w is None else w) + (0.0 if b is None else b)


def layer_norm_bwd(x, w, eps, gy):
    """(dx, the terms of dw, the terms of db), one term per row."""
    C = x.shape[-1]
    mu = x.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt(((x - mu) ** 2).mean(-1, keepdims=True) + eps)
    xh = (x - mu) * r
    t = gy * (1.0 if w is None else w)
    # the Jacobian of xh: r (I - 1/C - xh xh^T / C)
    dx = r * (t - t.sum(-1, keepdims=True) / C - xh * (t * xh).sum(-1, keepdims=True) / C)
    return dx, gy * xh, gy
