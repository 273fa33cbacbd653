"""fp64 definitions of the decayed linear attention, rotary positions and layer
norm (test infrastructure only, like the rest of this package; numpy).

Linear attention, token by token, per head h reading q, k of head h // (H / Hk):
  S_t = e^{g_t} S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t
Its gradient for L = <dO, o> + <dhT, hT> is the chain rule through that
recurrence in reverse, with every state kept.
"""
import numpy as np

from .layer_ops import _f64


def _setup(q, k, v, g, cu):
    q, k, v, g = _f64(q), _f64(k), _f64(v), _f64(g)
    T, Hk, d = q.shape
    H = v.shape[1]
    g = np.broadcast_to(g, (T, H)) if g.ndim == 1 else g
    return np.repeat(q, H // Hk, 1), np.repeat(k, H // Hk, 1), v, np.exp(g), [int(c) for c in cu], Hk


def linear_forward(q, k, v, g, cu_seqlens, h0=None, scale=1.0):
    """(o [T, H, d], hT [N, H, d, d])."""
    q, k, v, a, cu, _ = _setup(q, k, v, g, cu_seqlens)
    T, H, d = v.shape
    N = len(cu) - 1
    o = np.zeros((T, H, d))
    hT = np.zeros((N, H, d, d)) if h0 is None else _f64(h0).copy()
    for n in range(N):
        S = hT[n]
        for t in range(cu[n], cu[n + 1]):
            S = a[t][:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
            o[t] = scale * np.einsum("hij,hi->hj", S, q[t])
        hT[n] = S
    return o, hT


def linear_backward(q, k, v, g, dO, cu_seqlens, h0=None, dhT=None, scale=1.0):
    """dict of dq, dk [T, Hk, d], dv [T, H, d], dg (g's shape), dh0."""
    const = _f64(g).ndim == 1
    q, k, v, a, cu, Hk = _setup(q, k, v, g, cu_seqlens)
    dO = _f64(dO) * scale
    T, H, d = v.shape
    N = len(cu) - 1
    S0 = np.zeros((N, H, d, d)) if h0 is None else _f64(h0)
    dS = np.zeros((N, H, d, d)) if dhT is None else _f64(dhT).copy()
    dq, dk, dv, dg = np.zeros_like(q), np.zeros_like(q), np.zeros_like(v), np.zeros_like(a)
    for n in range(N):
        states = [S0[n]]
        for t in range(cu[n], cu[n + 1]):
            states.append(a[t][:, None, None] * states[-1] + k[t][:, :, None] * v[t][:, None, :])
        E = dS[n]
        for t in reversed(range(cu[n], cu[n + 1])):
            i = t - cu[n]
            dq[t] = np.einsum("hij,hj->hi", states[i + 1], dO[t])
            E = E + q[t][:, :, None] * dO[t][:, None, :]
            dk[t] = np.einsum("hij,hj->hi", E, v[t])
            dv[t] = np.einsum("hij,hi->hj", E, k[t])
            E = a[t][:, None, None] * E
            dg[t] = np.einsum("hij,hij->h", E, states[i])
        dS[n] = E
    share = lambda x: x.reshape(T, Hk, H // Hk, d).sum(2)
    return {"dq": share(dq), "dk": share(dk), "dv": dv, "dg": dg.sum(0) if const else dg, "dh0": dS}


def rotary(x, inv_freq, positions, interleaved=False, inverse=False, scale=1.0):
    """x [T, H, d], the first 2 len(inv_freq) channels turned."""
    x, f = _f64(x), _f64(inv_freq)
    half = f.shape[0]
    angle = _f64(positions)[:, None] * f[None, :] * (-1.0 if inverse else 1.0)
    turn = scale * np.exp(1j * angle)[:, None, :]
    y = x.copy()
    if interleaved:
        z = (x[..., 0:2 * half:2] + 1j * x[..., 1:2 * half:2]) * turn
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = z.real, z.imag
    else:
        z = (x[..., :half] + 1j * x[..., half:2 * half]) * turn
        y[..., :half], y[..., half:2 * half] = z.real, z.imag
    return y


def sequence_positions(cu_seqlens):
    cu = [int(c) for c in cu_seqlens]
    return np.concatenate([np.arange(b - a) for a, b in zip(cu[:-1], cu[1:])] or [np.zeros(0)])


def layernorm(x, weight=None, bias=None, eps=1e-5):
    """(y, mean, rstd) over the last axis."""
    x = _f64(x)
    m = x.mean(-1)
    r = 1.0 / np.sqrt(((x - m[..., None]) ** 2).mean(-1) + eps)
    y = (x - m[..., None]) * r[..., None]
    if weight is not None:
        y = y * _f64(weight)
    if bias is not None:
        y = y + _f64(bias)
    return y, m, r


def layernorm_backward(dy, x, weight=None, eps=1e-5, groups=1):
    """dict of dx, dweight, dbias; the sums run over all rows of [T, groups, D]
    of one group ([groups, D]), or all rows ([D]) for groups = 0."""
    dy, x = _f64(dy), _f64(x)
    _, m, r = layernorm(x, eps=eps)
    xh = (x - m[..., None]) * r[..., None]
    u = dy if weight is None else dy * _f64(weight)
    dx = r[..., None] * (u - u.mean(-1, keepdims=True) - xh * (u * xh).mean(-1, keepdims=True))
    D = x.shape[-1]
    shape = (-1, groups, D) if groups else (-1, D)
    return {"dx": dx, "dweight": (dy * xh).reshape(shape).sum(0), "dbias": dy.reshape(shape).sum(0)}
