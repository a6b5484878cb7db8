"""The gated delta rule in fp64, token by token, and its adjoint (test infrastructure; numpy).

    S~ = exp(log_a) S,  e = v - S~^T k,  u = beta e,  S = S~ + k u^T,  y = scale S^T q

All sequences of a packed batch run by themselves.
"""
from __future__ import annotations

import numpy as np


def _spans(cu):
    return [(int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])]


def forward(q, k, v, log_a, beta, cu, scale, init=None):
    """q, k [T,G,N], v [T,H,P], log_a, beta [T,H], init [n,H,N,P] -> y [T,H,P], final [n,H,N,P] (rows of no sequence zero)."""
    T, G, N = q.shape
    H, P = v.shape[1:]
    r = H // G
    y, finals = np.zeros((T, H, P)), np.zeros((len(cu) - 1, H, N, P))
    for s, (lo, hi) in enumerate(_spans(cu)):
        S = np.zeros((H, N, P)) if init is None else init[s].copy()
        for t in range(lo, hi):
            qt, kt = np.repeat(q[t], r, 0), np.repeat(k[t], r, 0)
            S = S * np.exp(log_a[t])[:, None, None]
            u = beta[t][:, None] * (v[t] - np.einsum("hnp,hn->hp", S, kt))
            S = S + kt[:, :, None] * u[:, None, :]
            y[t] = scale * np.einsum("hnp,hn->hp", S, qt)
        finals[s] = S
    return y, finals


def backward(q, k, v, log_a, beta, cu, scale, dy, init=None, dfinal=None):
    """Gradients of <dy, y> + <dfinal, final>: dq, dk [T,G,N], dv [T,H,P], dlog_a, dbeta [T,H], dinit [n,H,N,P]."""
    T, G, N = q.shape
    H, P = v.shape[1:]
    r, n = H // G, len(cu) - 1
    dq, dk, dv = np.zeros((T, H, N)), np.zeros((T, H, N)), np.zeros((T, H, P))
    dla, dbeta, dinit = np.zeros((T, H)), np.zeros((T, H)), np.zeros((n, H, N, P))
    for s, (lo, hi) in enumerate(_spans(cu)):
        S = np.zeros((H, N, P)) if init is None else init[s].copy()
        kept = []
        for t in range(lo, hi):
            kt = np.repeat(k[t], r, 0)
            old = S * np.exp(log_a[t])[:, None, None]
            e = v[t] - np.einsum("hnp,hn->hp", old, kt)
            S = old + kt[:, :, None] * (beta[t][:, None] * e)[:, None, :]
            kept.append((old, e, S))
        dS = np.zeros((H, N, P)) if dfinal is None else dfinal[s].copy()
        for t in reversed(range(lo, hi)):
            old, e, S = kept.pop()
            qt, kt = np.repeat(q[t], r, 0), np.repeat(k[t], r, 0)
            dq[t] = scale * np.einsum("hnp,hp->hn", S, dy[t])
            dS = dS + scale * qt[:, :, None] * dy[t][:, None, :]
            du = np.einsum("hnp,hn->hp", dS, kt)
            dbeta[t] = (du * e).sum(-1)
            dv[t] = beta[t][:, None] * du
            dk[t] = np.einsum("hnp,hp->hn", dS, beta[t][:, None] * e) - np.einsum("hnp,hp->hn", old, dv[t])
            dS = dS - kt[:, :, None] * dv[t][:, None, :]
            dla[t] = (dS * old).sum((-1, -2))
            dS = dS * np.exp(log_a[t])[:, None, None]
        dinit[s] = dS
    fold = lambda x: x.reshape(T, G, r, N).sum(2)  # noqa: E731
    return dict(dq=fold(dq), dk=fold(dk), dv=dv, dlog_a=dla, dbeta=dbeta, dinit=dinit)


def step(state, q, k, v, log_a, beta, scale):
    """One token each: state [n,H,N,P], q, k [n,G,N], v [n,H,P], log_a, beta [n,H] -> y, state."""
    cu = np.arange(len(v) + 1)
    return forward(q, k, v, log_a, beta, cu, scale, state)
