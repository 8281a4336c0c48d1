"""Plain fp64 CPU oracle of the layer norm with grouped affine weights.

TEST INFRASTRUCTURE ONLY (see ``oracle/ttt_oracle.py`` for the rules).

n = (r - mean(r)) / sqrt(var(r) + eps), y = n w_g + b_g with row i in group
(i / period) % groups; r = x, or x + res as the caller rounds it.  Next to each
value stands the bound on what fp32 arithmetic may add to it.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
# Roundings along one sum over a row: a thread adds at most 32 elements, a wave 6
# times, the workgroup 16 (rows up to 32768 elements).
SUM_OPS = 56.0


def groups_of(rows, groups, period):
    return (np.arange(rows) // period) % groups


def forward(r, w, b, eps, groups=1, period=1):
    """dict of y, n, mean, rstd and e_y, e_n, e_mean, e_rstd."""
    r = np.asarray(r, dtype=np.float64)
    g = groups_of(r.shape[0], groups, period)
    D = r.shape[1]
    w = np.ones((groups, D)) if w is None else np.asarray(w, dtype=np.float64)
    b = np.zeros((groups, D)) if b is None else np.asarray(b, dtype=np.float64)
    mean = r.mean(1, keepdims=True)
    xc = r - mean
    var = (xc * xc).mean(1, keepdims=True)
    s = 1.0 / np.sqrt(var + eps)
    n = xc * s
    y = n * w[g] + b[g]
    e_mean = SUM_OPS * U * np.abs(r).mean(1, keepdims=True)
    e_xc = e_mean + U * np.abs(xc)
    # d var = mean(2 |xc| e_xc) + the sum's own roundings; s = (var + eps)^(-1/2)
    e_var = (2 * np.abs(xc) * e_xc).mean(1, keepdims=True) + (e_mean ** 2) + (SUM_OPS + 2) * U * var
    e_s = s * (0.5 * e_var / (var + eps) + 6 * U)
    e_n = s * e_xc + np.abs(xc) * e_s + U * np.abs(n)
    e_y = np.abs(w[g]) * e_n + 2 * U * (np.abs(n * w[g]) + np.abs(b[g]))
    return dict(y=y, n=n, mean=mean[:, 0], rstd=s[:, 0], e_y=e_y, e_n=e_n, e_mean=e_mean[:, 0], e_rstd=e_s[:, 0])


def backward(r, w, eps, dy, dr=None, groups=1, period=1):
    """dict of dx, dw, db and e_dx, e_dw, e_db."""
    f = forward(r, w, None, eps, groups, period)
    dy = np.asarray(dy, dtype=np.float64)
    rows, D = dy.shape
    g = groups_of(rows, groups, period)
    w = np.ones((groups, D)) if w is None else np.asarray(w, dtype=np.float64)
    n, en, s, es = f["n"], f["e_n"], f["rstd"][:, None], f["e_rstd"][:, None]
    t = w[g] * dy
    m1, m2 = t.mean(1, keepdims=True), (t * n).mean(1, keepdims=True)
    core = t - m1 - n * m2
    dx = s * core
    e_m1 = (SUM_OPS + 2) * U * np.abs(t).mean(1, keepdims=True)
    e_m2 = (SUM_OPS + 2) * U * np.abs(t * n).mean(1, keepdims=True) + (np.abs(t) * en).mean(1, keepdims=True)
    e_core = e_m1 + np.abs(n) * e_m2 + np.abs(m2) * en + 4 * U * (np.abs(t) + np.abs(m1) + np.abs(n * m2))
    e_dx = s * e_core + np.abs(core) * es + U * np.abs(dx)
    if dr is not None:
        dx = dx + np.asarray(dr, dtype=np.float64)
        e_dx = e_dx + U * np.abs(dx)
    dw, db, e_dw, e_db = (np.zeros((groups, D)) for _ in range(4))
    for k in range(groups):
        at = g == k
        ops = (at.sum() + 1) * U  # one rounding a row, in whatever order
        dw[k], db[k] = (dy[at] * n[at]).sum(0), dy[at].sum(0)
        e_dw[k] = (np.abs(dy[at]) * en[at]).sum(0) + ops * np.abs(dy[at] * n[at]).sum(0)
        e_db[k] = ops * np.abs(dy[at]).sum(0)
    return dict(dx=dx, dw=dw, db=db, e_dx=e_dx, e_dw=e_dw, e_db=e_db)
