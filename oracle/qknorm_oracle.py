"""Plain fp64 CPU oracle of the norm and rotation of queries and keys.

TEST INFRASTRUCTURE ONLY (see ``oracle/ttt_oracle.py`` for the rules).

A row x of d values: h = x, x / sqrt(mean(x^2) + eps) ("rms") or
x / sqrt(sum(x^2) + eps) ("l2"); z = w h; then pair j of the first 2 len(freq)
columns, (j, j + len(freq)) ("half") or (2 j, 2 j + 1) ("interleaved"), turns by
pos * freq_j, times ``scale``.
"""
from __future__ import annotations

import numpy as np


def _pairs(half, pairing):
    j = np.arange(half)
    return (j, j + half) if pairing == "half" else (2 * j, 2 * j + 1)


def turn(x, pos, freq, pairing, scale=1.0, back=False):
    """[tokens, H, d] with each token's pairs turned."""
    freq = np.asarray(freq, dtype=np.float64)
    angle = np.asarray(pos, dtype=np.float64)[:, None, None] * freq
    c, s = scale * np.cos(angle), scale * np.sin(angle) * (-1.0 if back else 1.0)
    a, b = _pairs(len(freq), pairing)
    y = np.array(x, dtype=np.float64)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return y


def _hat(x, norm, eps):
    """x / size and 1 / size; a row of zeros is 0 / 0 where eps is zero."""
    ss = (x * x).sum(-1, keepdims=True)
    if norm == "none":
        return x, np.ones_like(ss)
    with np.errstate(divide="ignore", invalid="ignore"):
        r = 1.0 / np.sqrt((ss / x.shape[-1] if norm == "rms" else ss) + eps)
        return x * r, r


def forward(x, w, pos, freq, norm, pairing, eps=1e-6, scale=1.0):
    x = np.asarray(x, dtype=np.float64)
    h, _ = _hat(x, norm, eps)
    return turn(h if w is None else h * np.asarray(w, dtype=np.float64), pos, freq, pairing, scale)


def backward(x, w, pos, freq, norm, pairing, dy, eps=1e-6, scale=1.0):
    """dx, dw."""
    x = np.asarray(x, dtype=np.float64)
    h, r = _hat(x, norm, eps)
    dz = turn(np.asarray(dy, dtype=np.float64), pos, freq, pairing, scale, back=True)
    dw = (dz * h).sum((0, 1))
    dh = dz if w is None else dz * np.asarray(w, dtype=np.float64)
    dot = (dh * h).sum(-1, keepdims=True) / (x.shape[-1] if norm == "rms" else 1)
    return (dh if norm == "none" else r * (dh - h * dot)), dw
