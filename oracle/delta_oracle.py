"""Plain fp64 CPU oracle of the gated delta rule.

TEST INFRASTRUCTURE ONLY (see ``oracle/ttt_oracle.py`` for the rules).

Per sequence and value head, token by token: S <- a S; e = v - S^T k;
S <- S + eta k e^T; o = scale S^T q, with a = sigmoid(gate), exp(gate) or 1 and
eta = lr_max sigmoid(beta + lr_bias).  Sequences lie behind one another on one
token axis; ``starts`` holds their first rows and the end of the last.
"""
from __future__ import annotations

import numpy as np


def _sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def coefficients(gate, beta, kind, lr_max=1.0, lr_bias=0.0):
    """a, da/dgate, eta, deta/dbeta."""
    b = np.asarray(beta, dtype=np.float64) + lr_bias
    eta, deta = lr_max * _sigmoid(b), lr_max * _sigmoid(b) * _sigmoid(-b)
    if gate is None:
        return np.ones_like(b), np.zeros_like(b), eta, deta
    z = np.asarray(gate, dtype=np.float64)
    if kind == "sigmoid":
        return _sigmoid(z), _sigmoid(z) * _sigmoid(-z), eta, deta
    return np.exp(z), np.exp(z), eta, deta


def _heads(x, H):
    x = np.asarray(x, dtype=np.float64)
    return np.repeat(x, H // x.shape[1], axis=1)


def forward(q, k, v, gate, beta, starts, kind, scale, s0=None, lr_max=1.0, lr_bias=0.0):
    """(o [n,H,dv], s_final [B,H,dk,dv]); q, k [n,Hk,dk], v [n,H,dv], gate (or None), beta [n,H]."""
    v = np.asarray(v, dtype=np.float64)
    n, H, dv = v.shape
    q, k = _heads(q, H), _heads(k, H)
    a, _, eta, _ = coefficients(gate, beta, kind, lr_max, lr_bias)
    B = len(starts) - 1
    final = np.zeros((B, H, q.shape[2], dv)) if s0 is None else np.array(s0, dtype=np.float64)
    o = np.zeros((n, H, dv))
    for s in range(B):
        S = final[s]
        for t in range(starts[s], starts[s + 1]):
            S = a[t][:, None, None] * S
            e = v[t] - np.einsum("hij,hi->hj", S, k[t])
            S = S + np.einsum("hi,hj->hij", k[t], eta[t][:, None] * e)
            o[t] = scale * np.einsum("hij,hi->hj", S, q[t])
        final[s] = S
    return o, final


def backward(q, k, v, gate, beta, starts, kind, scale, d_o, s0=None, d_sfinal=None, lr_max=1.0, lr_bias=0.0):
    """dict of dq, dk, dv, dgate, dbeta, ds0 for <d_o, o> + <d_sfinal, s_final>, by the chain rule of each token."""
    v = np.asarray(v, dtype=np.float64)
    n, H, dv = v.shape
    Hk, dk = np.shape(q)[1:]
    qh, kh = _heads(q, H), _heads(k, H)
    d_o = np.asarray(d_o, dtype=np.float64)
    a, da, eta, deta = coefficients(gate, beta, kind, lr_max, lr_bias)
    B = len(starts) - 1
    S0 = np.zeros((B, H, dk, dv)) if s0 is None else np.asarray(s0, dtype=np.float64)
    dS0 = np.zeros((B, H, dk, dv)) if d_sfinal is None else np.array(d_sfinal, dtype=np.float64)
    dq, dk_, dv_ = np.zeros((n, H, dk)), np.zeros((n, H, dk)), np.zeros((n, H, dv))
    dgate, dbeta = np.zeros((n, H)), np.zeros((n, H))
    for s in range(B):
        S, trace = S0[s], []
        for t in range(starts[s], starts[s + 1]):
            old = a[t][:, None, None] * S
            e = v[t] - np.einsum("hij,hi->hj", old, kh[t])
            new = old + np.einsum("hi,hj->hij", kh[t], eta[t][:, None] * e)
            trace.append((S, old, e, new))
            S = new
        dS = dS0[s]
        for t in range(starts[s + 1] - 1, starts[s] - 1, -1):
            first, old, e, new = trace[t - starts[s]]
            dS = dS + scale * np.einsum("hi,hj->hij", qh[t], d_o[t])
            dq[t] = scale * np.einsum("hij,hj->hi", new, d_o[t])
            toward = np.einsum("hij,hi->hj", dS, kh[t])
            dbeta[t] = (toward * e).sum(-1) * deta[t]
            de = eta[t][:, None] * toward
            dv_[t] = de
            dk_[t] = np.einsum("hij,hj->hi", dS, eta[t][:, None] * e) - np.einsum("hij,hj->hi", old, de)
            dS = dS - np.einsum("hi,hj->hij", kh[t], de)
            dgate[t] = (dS * first).sum((1, 2)) * da[t]
            dS = a[t][:, None, None] * dS
        dS0[s] = dS
    return dict(dq=dq.reshape(n, Hk, -1, dk).sum(2), dk=dk_.reshape(n, Hk, -1, dk).sum(2), dv=dv_, dgate=dgate, dbeta=dbeta,
                ds0=dS0)
