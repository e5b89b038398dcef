"""FP64 oracle of the gated delta rule with one decay per head and token, token by
token from its definition, with its hand-derived adjoint; of the verification of
drafted tokens; and of the layer norm.

Token tensors are [B, T, H, 128], gates [B, T, H]; `lengths` and `packed` describe
the sequences as in kda_oracle.  NumPy only.
"""
from __future__ import annotations

import numpy as np

from .layer_oracle import _f64, _spans

NORM_EPS = 1e-6


def _unit(x, on):
    size = np.sqrt((x * x).sum(-1, keepdims=True) + NORM_EPS) if on else np.ones_like(x[..., :1])
    return x / size, size


def delta_forward(q, k, v, g, beta, state, lengths, packed, scale, unit):
    """(o, final state, weights): S <- e^g S, S <- S + beta (v - S k) k^T, o = scale S q.

    `weights` bounds the sizes of what the sums hold, row by row of the state, for
    the bars of a comparison: (of o, of the final state), from N <- e^g N + |beta w| |k|
    with the written rows w = v - S k themselves (|k| the 2-norm), N starting as the
    rows' 2-norms, and of the final state M <- e^g M + |beta| (|v| + N |k|) |k|: what the
    written rows are made of, each as large as its terms rather than as their sum."""
    q, k, v, g, beta, state = map(_f64, (q, k, v, g, beta, state))
    G = v.shape[2] // q.shape[2]
    (q, _), (k, _) = _unit(q, unit), _unit(k, unit)
    o, wo = np.zeros_like(v), np.zeros_like(v)
    final, wfinal, states = np.zeros_like(state), np.zeros(state.shape[:3]), {}
    for n, (b, t0, L) in enumerate(_spans(lengths, packed, q.shape[1])):
        S = state[n].copy()
        N = np.linalg.norm(S, axis=-1)
        M = N.copy()
        for t in range(t0, t0 + L):
            kt, qt = np.repeat(k[b, t], G, 0), np.repeat(q[b, t], G, 0)
            a, bt = np.exp(g[b, t])[:, None], beta[b, t][:, None]
            nk, nq = np.linalg.norm(kt, axis=-1)[:, None], np.linalg.norm(qt, axis=-1)[:, None]
            S = a[..., None] * S
            N, M = a * N, a * M
            w = v[b, t] - np.einsum("hvk,hk->hv", S, kt)
            S = S + (bt * w)[:, :, None] * kt[:, None, :]
            M = M + np.abs(bt) * (np.abs(v[b, t]) + N * nk) * nk
            N = N + np.abs(bt * w) * nk
            o[b, t] = scale * np.einsum("hvk,hk->hv", S, qt)
            wo[b, t] = scale * M * nq
            states[n, t - t0] = S
        final[n], wfinal[n] = S, M
    return o, final, (wo, wfinal), states


def delta_backward(q, k, v, g, beta, state, do, dfinal, lengths, packed, scale, unit):
    """((dq, dk, dv, dg, dbeta, dinitial), weights, parts) of <do, o> + <dfinal, final
    state>, by the adjoint of the recurrence: with Z the state's adjoint,
        Z += scale do q^T;  u = Z k;  dbeta = u.w;  dv = beta u;
        dq = scale S^T do;  dk = beta Z^T w - beta X^T u  (X the decayed state before);
        Z -= beta u k^T;  dg = <Z, X>;  Z <- e^g Z.
    `weights` bounds the sizes of what each gradient's sums hold: M of the state's rows as in
    delta_forward, and for Z's rows NZ <- NZ + scale |do| |q| + |beta u| |k| and MZ <- MZ + scale
    |do| |q| + |beta| NZ |k|^2, both decaying with Z (of the last, dinitial, per row).  `parts`: for
    dq and dk the sums over the value heads of their absolute parts."""
    q, k, v, g, beta, state, do, dfinal = map(_f64, (q, k, v, g, beta, state, do, dfinal))
    Hqk = q.shape[2]
    G = v.shape[2] // Hqk
    (q, nq), (k, nk) = _unit(q, unit), _unit(k, unit)
    grads = dq, dk, dv, dg, dbeta = [np.zeros_like(x) for x in (q, k, v, g, beta)]
    weights = wq, wk, wv, wg, wb = [np.zeros_like(x) for x in grads]
    pq, pk = np.zeros_like(q), np.zeros_like(k)
    dinit, winit = np.zeros_like(state), np.zeros(state.shape[:3])
    shared = lambda x: x.reshape(Hqk, G, -1).sum(1)  # noqa: E731
    for n, (b, t0, L) in enumerate(_spans(lengths, packed, q.shape[1])):
        S, X = state[n].copy(), []
        N = M = np.linalg.norm(S, axis=-1)
        for t in range(t0, t0 + L):
            kt, a, bt = np.repeat(k[b, t], G, 0), np.exp(g[b, t])[:, None], beta[b, t][:, None]
            nkt = np.linalg.norm(kt, axis=-1)[:, None]
            S, N, M = a[..., None] * S, a * N, a * M
            X.append((S, M))
            w = v[b, t] - np.einsum("hvk,hk->hv", S, kt)
            S = S + (bt * w)[:, :, None] * kt[:, None, :]
            M = M + np.abs(bt) * (np.abs(v[b, t]) + N * nkt) * nkt
            N = N + np.abs(bt * w) * nkt
        Z = dfinal[n].copy()
        NZ = MZ = np.linalg.norm(Z, axis=-1)
        for t in reversed(range(t0, t0 + L)):
            kt, qt, bt, (x, m) = np.repeat(k[b, t], G, 0), np.repeat(q[b, t], G, 0), beta[b, t][:, None], X[t - t0]
            nkt, nqt = (np.linalg.norm(y, axis=-1)[:, None] for y in (kt, qt))
            w = v[b, t] - np.einsum("hvk,hk->hv", x, kt)
            after = x + (bt * w)[:, :, None] * kt[:, None, :]
            d = scale * do[b, t]
            Z, NZ, MZ = Z + d[:, :, None] * qt[:, None, :], NZ + np.abs(d) * nqt, MZ + np.abs(d) * nqt
            u = np.einsum("hvk,hk->hv", Z, kt)
            gq = np.einsum("hvk,hv->hk", after, d)
            gk = np.einsum("hvk,hv->hk", Z, bt * w) - np.einsum("hvk,hv->hk", x, bt * u)
            dbeta[b, t], dv[b, t] = (u * w).sum(-1), bt * u
            mw = np.abs(v[b, t]) + m * nkt               # sizes of w's terms
            ma = m + np.abs(bt) * mw * nkt               # of the state behind the token
            cq = (ma * np.abs(d)).sum(-1, keepdims=True)
            ck = (np.abs(bt) * (MZ * mw + m * MZ * nkt)).sum(-1, keepdims=True)
            wb[b, t], wv[b, t] = (MZ * nkt * mw).sum(-1), np.abs(bt) * MZ * nkt
            Z = Z - (bt * u)[:, :, None] * kt[:, None, :]
            MZ = MZ + np.abs(bt) * NZ * nkt * nkt
            NZ = NZ + np.abs(bt * u) * nkt
            dg[b, t], wg[b, t] = (Z * x).sum((-1, -2)), (MZ * m).sum(-1)
            a = np.exp(g[b, t])[:, None]
            Z, NZ, MZ = a[..., None] * Z, a * NZ, a * MZ
            if unit:
                sq, sk = np.repeat(nq[b, t], G, 0), np.repeat(nk[b, t], G, 0)
                gq, gk = ((y - hat * (y * hat).sum(-1, keepdims=True)) / size for y, hat, size in ((gq, qt, sq), (gk, kt, sk)))
                cq, ck = cq / sq, ck / sk
            dq[b, t], dk[b, t] = shared(gq), shared(gk)
            wq[b, t], wk[b, t] = shared(cq), shared(ck)
            pq[b, t], pk[b, t] = shared(np.abs(gq)), shared(np.abs(gk))
        dinit[n], winit[n] = Z, MZ
    return (*grads, dinit), (*weights, winit), (pq, pk)


def verify(drafts, lens, target, draft, uniform):
    """(tokens, number accepted): draft i stands while u_i q(x_i) < p(x_i); then one
    draw from the positive part of p - q, from p behind the last draft or where that
    part is zero."""
    target, uniform = _f64(target), _f64(uniform)
    N, S = drafts.shape
    V = target.shape[2]
    tokens, accepted = np.full((N, S + 1), -1, np.int32), np.zeros(N, np.int32)
    for n in range(N):
        L = S if lens is None else min(max(int(lens[n]), 0), S)
        j = 0
        while j < L:
            x = int(drafts[n, j])
            if not 0 <= x < V:
                break
            qx = 1.0 if draft is None else float(draft[n, j, x])
            if not uniform[n, j] * qx < target[n, j, x]:
                break
            tokens[n, j] = x
            j += 1
        p = target[n, j]
        w = p.copy()
        if j < L:
            if draft is not None:
                w = p - _f64(draft[n, j])
            elif 0 <= int(drafts[n, j]) < V:
                w[int(drafts[n, j])] = 0.0
        w = np.where(w > 0, w, 0.0)
        if not w.sum() > 0:
            w = np.where(p > 0, p, 0.0)
        run = np.cumsum(w)
        if run[-1] > 0:
            u = uniform[n, S]
            past = np.flatnonzero((run > (u if u > 0 else 0.0) * run[-1]) & (w > 0))
            tokens[n, j] = past[0] if len(past) else np.flatnonzero(w > 0)[-1]
        accepted[n] = j + 1
    return tokens, accepted


def layer_norm(x, w, b, eps):
    x, w = _f64(x), _f64(w)
    hat = x - x.mean(-1, keepdims=True)
    hat = hat / np.sqrt((hat * hat).mean(-1, keepdims=True) + eps)
    return hat * w + (0.0 if b is None else _f64(b)), hat


def layer_norm_backward(dy, x, w, eps):
    """(dx, dw, db)."""
    dy, x, w = map(_f64, (dy, x, w))
    m = x - x.mean(-1, keepdims=True)
    size = np.sqrt((m * m).mean(-1, keepdims=True) + eps)
    hat, d = m / size, dy * w
    dx = (d - d.mean(-1, keepdims=True) - hat * (d * hat).mean(-1, keepdims=True)) / size
    return dx, (dy * hat).sum(0), dy.sum(0)
