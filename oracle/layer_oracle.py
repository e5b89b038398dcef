"""FP64 oracle of the linear-attention layer operators, from their definitions:
linear attention with a constant decay per head, token by token, with its
hand-derived adjoint; the query/key norm with rotary rotation; the gated norm.

Token tensors are [B, T, H, 128]; `lengths` and `packed` describe the
sequences as in kda_oracle.  NumPy only.
"""
from __future__ import annotations

import numpy as np

D = 128


def _f64(x):
    return np.asarray(x, dtype=np.float64)


def _spans(lengths, packed, T):
    """(batch row, first token, length) of every sequence."""
    if not packed:
        return [(b, 0, L) for b, L in enumerate(lengths)]
    out, at = [], 0
    for L in lengths:
        out.append((0, at, L))
        at += L
    return out


def decay_forward(q, k, v, log_decay, state, lengths, packed, scale):
    """(o, final state, majorants of |o| and of |final state|): S <- e^l S + v k^T,
    o = scale S q.  The majorants are the same recurrence over absolute values."""
    q, k, v, state = map(_f64, (q, k, v, state))
    lam = np.exp(_f64(log_decay))[:, None, None]
    G = v.shape[2] // q.shape[2]
    o, major, final, mfinal = np.zeros_like(v), np.zeros_like(v), np.zeros_like(state), np.zeros_like(state)
    for n, (b, t0, L) in enumerate(_spans(lengths, packed, q.shape[1])):
        S, M = state[n].copy(), np.abs(state[n])
        for t in range(t0, t0 + L):
            kt, qt = np.repeat(k[b, t], G, 0), np.repeat(q[b, t], G, 0)
            S = lam * S + v[b, t][:, :, None] * kt[:, None, :]
            M = lam * M + np.abs(v[b, t][:, :, None] * kt[:, None, :])
            o[b, t] = scale * np.einsum("hvk,hk->hv", S, qt)
            major[b, t] = scale * np.einsum("hvk,hk->hv", M, np.abs(qt))
        final[n], mfinal[n] = S, M
    return o, final, major, mfinal


def decay_backward(q, k, v, log_decay, state, do, dfinal, lengths, packed, scale):
    """(dq, dk, dv, dinitial) of <do, o> + <dfinal, final state>."""
    q, k, v, state, do, dfinal = map(_f64, (q, k, v, state, do, dfinal))
    lam = np.exp(_f64(log_decay))[:, None, None]
    Hqk = q.shape[2]
    G = v.shape[2] // Hqk
    dq, dk, dv, dinit = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros_like(state)
    shared = lambda x: x.reshape(Hqk, G, D).sum(1)  # noqa: E731
    for n, (b, t0, L) in enumerate(_spans(lengths, packed, q.shape[1])):
        S = state[n].copy()
        for t in range(t0, t0 + L):
            S = lam * S + v[b, t][:, :, None] * np.repeat(k[b, t], G, 0)[:, None, :]
            dq[b, t] = shared(scale * np.einsum("hvk,hv->hk", S, do[b, t]))
        dS = dfinal[n].copy()
        for t in reversed(range(t0, t0 + L)):
            kt, qt = np.repeat(k[b, t], G, 0), np.repeat(q[b, t], G, 0)
            dS = dS + scale * do[b, t][:, :, None] * qt[:, None, :]
            dk[b, t] = shared(np.einsum("hvk,hv->hk", dS, v[b, t]))
            dv[b, t] = np.einsum("hvk,hk->hv", dS, kt)
            dS = lam * dS
        dinit[n] = dS
    return dq, dk, dv, dinit


def _rotation(cos, sin, positions, rot, pairs):
    """[B, T, 128, 128] rotation matrices."""
    B, T = positions.shape
    R = np.zeros((B, T, D, D))
    R[:] = np.eye(D)
    p = np.arange(rot // 2)
    u, v = (2 * p, 2 * p + 1) if pairs else (p, p + rot // 2)
    c, s = _f64(cos)[positions], _f64(sin)[positions]
    R[:, :, u, u], R[:, :, v, v] = c, c
    R[:, :, u, v], R[:, :, v, u] = -s, s
    return R


def qk_norm_rope(x, w, cos, sin, positions, rot, pairs, eps):
    x, w = _f64(x), _f64(w)
    n = w * x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return np.einsum("btij,bthj->bthi", _rotation(cos, sin, positions, rot, pairs), n)


def qk_norm_rope_backward(dy, x, w, cos, sin, positions, rot, pairs, eps):
    """(dx, dw)."""
    dy, x, w = map(_f64, (dy, x, w))
    dn = np.einsum("btij,bthi->bthj", _rotation(cos, sin, positions, rot, pairs), dy)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    g = dn * w
    dx = r * g - x * r ** 3 * (g * x).mean(-1, keepdims=True)
    return dx, (dn * x * r).sum((0, 1, 2))


def _act(g, silu):
    s = 1 / (1 + np.exp(-g))
    return (g * s, s * (1 + g * (1 - s))) if silu else (s, s * (1 - s))


def gated_norm(x, g, w, silu, eps):
    x, g, w = map(_f64, (x, g, w))
    return w * x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * _act(g, silu)[0]


def gated_norm_backward(dy, x, g, w, silu, eps):
    """(dx, dg, dw)."""
    dy, x, g, w = map(_f64, (dy, x, g, w))
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    a, slope = _act(g, silu)
    u = dy * w * a
    dx = r * u - x * r ** 3 * (u * x).mean(-1, keepdims=True)
    return dx, dy * w * x * r * slope, (dy * a * x * r).sum((0, 1, 2))
