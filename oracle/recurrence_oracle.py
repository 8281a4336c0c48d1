"""Plain fp64 CPU oracle of the gated linear recurrence.

TEST INFRASTRUCTURE ONLY (see ``oracle/ttt_oracle.py`` for the rules).

Per channel, h_t = a_t h_{t-1} + u_t with a = sigmoid(z) ("sigmoid") or exp(z)
("log") and u = x ("plain") or (1 - a) x ("convex"), from h0 of each sequence.
Sequences lie behind one another on one token axis; ``starts`` holds their first
rows and the end of the last.  Everything is a loop over tokens.

``error`` runs the same loops over magnitudes: the bound on what fp32 arithmetic
may add to each value, with every operation off by half a step.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # half a step of fp32, relative
# Operations on a value per token, each off by at most U of it: a = sigmoid(z) or
# exp(z) is off by the hardware exp2's and reciprocal's step (2 U each), the two
# sums and roundings of the argument (|z log2 e| U, |z| <= 12 in the tests, which
# e^-z / (1 + e^-z) or a fast decay damps, 18 U) and the multiply-add (2 U); the tile
# and wave maps round each value once more.
STEP_OPS = 26.0


def coefficients(z, gate):
    """a, 1 - a, da/dz."""
    z = np.asarray(z, dtype=np.float64)
    with np.errstate(over="ignore"):
        if gate == "sigmoid":
            a, rest = 1.0 / (1.0 + np.exp(-z)), 1.0 / (1.0 + np.exp(z))
            return a, rest, a * rest
        a = np.exp(z)
        return a, -np.expm1(z), a


def dense_starts(B, T):
    return np.arange(B + 1) * T


def forward(x, z, starts, gate, inp, h0=None):
    """(o [n, D], h_final [B, D], bound on o's fp32 error, bound on h_final's)."""
    a, rest, _ = coefficients(z, gate)
    u = np.asarray(x, dtype=np.float64) * (rest if inp == "convex" else 1.0)
    n, D = u.shape
    B = len(starts) - 1
    h0 = np.zeros((B, D)) if h0 is None else np.asarray(h0, dtype=np.float64)
    o, eo = np.zeros((n, D)), np.zeros((n, D))
    final, ef = h0.copy(), np.zeros((B, D))
    for s in range(B):
        h, m, e = h0[s], np.abs(h0[s]), np.zeros(D)
        for t in range(starts[s], starts[s + 1]):
            h = a[t] * h + u[t]
            m = a[t] * m + np.abs(u[t])
            e = a[t] * e + STEP_OPS * U * m
            o[t], eo[t] = h, e
        final[s], ef[s] = h, e
    return o, final, eo, ef


def backward(x, z, starts, gate, inp, d_o, h0=None, d_hfinal=None):
    """dict of dx, dgate, dh0, and the bounds on their fp32 errors under "e_" + name."""
    a, rest, da = coefficients(z, gate)
    x = np.asarray(x, dtype=np.float64)
    d_o = np.asarray(d_o, dtype=np.float64)
    n, D = x.shape
    B = len(starts) - 1
    o, _, eo, _ = forward(x, z, starts, gate, inp, h0)
    h0 = np.zeros((B, D)) if h0 is None else np.asarray(h0, dtype=np.float64)
    dh0 = np.zeros((B, D)) if d_hfinal is None else np.array(d_hfinal, dtype=np.float64)
    dx, dz = np.zeros((n, D)), np.zeros((n, D))
    edx, edz, edh0 = np.zeros((n, D)), np.zeros((n, D)), np.zeros((B, D))
    f = rest if inp == "convex" else np.ones_like(a)
    for s in range(B):
        g = dh0[s].copy()  # the gradient that reaches h_t from the tokens after t
        m, e = np.abs(g), np.zeros(D)
        for t in range(starts[s + 1] - 1, starts[s] - 1, -1):
            first = t == starts[s]
            before, eb = (h0[s], np.zeros(D)) if first else (o[t - 1], eo[t - 1])
            dh, m = d_o[t] + g, np.abs(d_o[t]) + m
            e = e + 2 * U * m
            w = before - x[t] if inp == "convex" else before
            size = np.abs(before) + (np.abs(x[t]) if inp == "convex" else 0.0)
            dx[t], dz[t] = dh * f[t], dh * da[t] * w
            edx[t] = e * f[t] + STEP_OPS * U * np.abs(dx[t])
            edz[t] = np.abs(da[t]) * (e * np.abs(w) + np.abs(dh) * (eb + STEP_OPS * U * size))
            g, m = a[t] * dh, a[t] * m
            e = a[t] * e + STEP_OPS * U * m
        dh0[s], edh0[s] = g, e
    return dict(dx=dx, dgate=dz, dh0=dh0, e_dx=edx, e_dgate=edz, e_dh0=edh0)
