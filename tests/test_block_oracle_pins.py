"""Pins of the recurrence and layer norm oracles (CPU): closed forms, finite
differences, and planted mistakes that the tolerances have to catch."""
import numpy as np
import pytest

from oracle import layernorm_oracle as ln
from oracle import recurrence_oracle as rec
from tests.block_utils import worst


@pytest.fixture
def rng():
    return np.random.default_rng(2024)


def _inputs(rng, n, D, B):
    return (rng.standard_normal((n, D)), rng.normal(1.0, 1.5, (n, D)), rng.standard_normal((B, D)),
            rng.standard_normal((n, D)), rng.standard_normal((B, D)))


@pytest.mark.parametrize("gate", ["sigmoid", "log"])
@pytest.mark.parametrize("inp", ["plain", "convex"])
def test_recurrence_is_the_weighted_sum_of_its_inputs(rng, gate, inp):
    x, z, h0, _, _ = _inputs(rng, 12, 3, 1)
    if gate == "log":
        z = -np.abs(z)
    o, final, _, _ = rec.forward(x, z, [0, 12], gate, inp, h0)
    a = 1 / (1 + np.exp(-z)) if gate == "sigmoid" else np.exp(z)
    u = x * (1 - a) if inp == "convex" else x
    for t in range(12):
        want = np.prod(a[:t + 1], 0) * h0[0] + sum(np.prod(a[s + 1:t + 1], 0) * u[s] for s in range(t + 1))
        assert np.allclose(o[t], want, rtol=1e-12, atol=1e-12)
    assert np.array_equal(final[0], o[-1])


def test_recurrence_sequences_are_independent_and_resume(rng):
    x, z, h0, d_o, dhf = _inputs(rng, 20, 4, 3)
    starts = [0, 7, 7, 20]
    o, final, _, _ = rec.forward(x, z, starts, "sigmoid", "convex", h0)
    assert np.array_equal(final[1], h0[1])  # an empty sequence passes its state on
    part, mid, _, _ = rec.forward(x[7:12], z[7:12], [0, 5], "sigmoid", "convex", h0[2:])
    rest, end, _, _ = rec.forward(x[12:20], z[12:20], [0, 8], "sigmoid", "convex", mid)
    assert np.allclose(np.concatenate([part, rest]), o[7:20]) and np.allclose(end[0], final[2])
    g = rec.backward(x, z, starts, "sigmoid", "convex", d_o, h0, dhf)
    assert np.array_equal(g["dh0"][1], dhf[1])


@pytest.mark.parametrize("gate", ["sigmoid", "log"])
@pytest.mark.parametrize("inp", ["plain", "convex"])
def test_recurrence_backward_finite_differences(rng, gate, inp):
    n, D, starts = 9, 2, [0, 4, 4, 9]
    x, z, h0, d_o, dhf = _inputs(rng, n, D, 3)
    z = -np.abs(z) if gate == "log" else z

    def loss(x_, z_, h_):
        o, f, _, _ = rec.forward(x_, z_, starts, gate, inp, h_)
        return (o * d_o).sum() + (f * dhf).sum()

    g = rec.backward(x, z, starts, gate, inp, d_o, h0, dhf)
    for name, k in (("dx", 0), ("dgate", 1), ("dh0", 2)):
        args = [x, z, h0]
        num = np.zeros_like(args[k])
        for at in np.ndindex(*args[k].shape):
            hi, lo = [v.copy() for v in args], [v.copy() for v in args]
            hi[k][at] += 1e-5
            lo[k][at] -= 1e-5
            num[at] = (loss(*hi) - loss(*lo)) / 2e-5
        assert np.allclose(num, g[name], rtol=1e-6, atol=1e-7), name


def test_recurrence_tolerance_catches_planted_mistakes(rng):
    x, z, h0, _, _ = _inputs(rng, 300, 8, 1)
    z += 3.0
    o, final, eo, _ = rec.forward(x, z, [0, 300], "sigmoid", "convex", h0)
    assert worst(o, o, eo, "bf16") == 0.0
    # the gate of the token before, the state not carried over a tile border, one token left out
    assert worst(rec.forward(x, np.roll(z, 1, 0), [0, 300], "sigmoid", "convex", h0)[0], o, eo, "bf16") > 10
    assert worst(rec.forward(x, z, [0, 128, 300], "sigmoid", "convex", np.repeat(h0, 2, 0))[0], o, eo, "bf16") > 10
    skip = x.copy()
    skip[200] = 0
    assert worst(rec.forward(skip, z, [0, 300], "sigmoid", "convex", h0)[0], o, eo, "bf16") > 2
    # a relative error of 1e-4 in fp32
    assert worst(o * (1 + 1e-4), o, eo, "f32") > 5


def test_layernorm_rows_are_normalised(rng):
    r = rng.standard_normal((6, 40)) * 5 + 3
    f = ln.forward(r, None, None, 0.0)
    assert np.allclose(f["y"].mean(1), 0) and np.allclose((f["y"] ** 2).mean(1), 1)
    w, b = rng.standard_normal((2, 40)), rng.standard_normal((2, 40))
    f = ln.forward(r, w, b, 1e-5, groups=2, period=3)
    for i in range(6):
        k = (i // 3) % 2
        want = (r[i] - r[i].mean()) / np.sqrt(r[i].var() + 1e-5) * w[k] + b[k]
        assert np.allclose(f["y"][i], want, rtol=1e-12)


def test_layernorm_backward_finite_differences(rng):
    r, w, b = rng.standard_normal((4, 5)), rng.standard_normal((2, 5)), rng.standard_normal((2, 5))
    dy, dr = rng.standard_normal((4, 5)), rng.standard_normal((4, 5))

    def loss(r_, w_, b_):
        return (ln.forward(r_, w_, b_, 1e-3, 2, 1)["y"] * dy).sum() + (r_ * dr).sum()

    g = ln.backward(r, w, 1e-3, dy, dr, 2, 1)
    for name, k in (("dx", 0), ("dw", 1), ("db", 2)):
        args = [r, w, b]
        num = np.zeros_like(args[k])
        for at in np.ndindex(*args[k].shape):
            hi, lo = [v.copy() for v in args], [v.copy() for v in args]
            hi[k][at] += 1e-5
            lo[k][at] -= 1e-5
            num[at] = (loss(*hi) - loss(*lo)) / 2e-5
        assert np.allclose(num, g[name], rtol=1e-6, atol=1e-7), name


def test_layernorm_tolerance_catches_planted_mistakes(rng):
    r, w, dy = rng.standard_normal((64, 100)), rng.standard_normal((2, 100)), rng.standard_normal((64, 100))
    f, g = ln.forward(r, w, None, 1e-5, 2, 16), ln.backward(r, w, 1e-5, dy, None, 2, 16)
    # the other group's weight, the unbiased variance, a gradient without its mean term, a row left out of dw
    assert worst(ln.forward(r, w[::-1], None, 1e-5, 2, 16)["y"], f["y"], f["e_y"], "bf16") > 10
    assert worst(f["y"] * np.sqrt(99 / 100), f["y"], f["e_y"], "f32") > 10
    bad = g["dx"] + f["rstd"][:, None] * (w[ln.groups_of(64, 2, 16)] * dy).mean(1, keepdims=True)
    assert worst(bad, g["dx"], g["e_dx"], "bf16") > 2
    part = ln.backward(r, w, 1e-5, np.concatenate([dy[:63], 0 * dy[63:]]), None, 2, 16)
    assert worst(part["dw"], g["dw"], g["e_dw"], "f32") > 10
