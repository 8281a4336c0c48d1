"""Pins of the gated delta rule's and the query and key norm's oracles (CPU): other oracles,
closed forms, finite differences."""
import numpy as np
import pytest

from oracle import chunk_forward
from oracle import delta_oracle as dr
from oracle import qknorm_oracle as qk


@pytest.fixture
def rng():
    return np.random.default_rng(77)


def _inputs(rng, n, H, Hk, dk, dv, B):
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)  # noqa: E731
    return dict(q=rng.standard_normal((n, Hk, dk)), k=unit(rng.standard_normal((n, Hk, dk))), v=rng.standard_normal((n, H, dv)),
                gate=rng.normal(1.0, 1.0, (n, H)), beta=rng.standard_normal((n, H)), s0=rng.standard_normal((B, H, dk, dv)))


def test_without_decay_it_is_the_fast_weight_layer_with_a_step_a_token(rng):
    x = _inputs(rng, 23, 2, 2, 5, 4, 1)
    o, final = dr.forward(x["q"], x["k"], x["v"], None, x["beta"], [0, 23], "sigmoid", 1.0, x["s0"], lr_max=2.0, lr_bias=-1.0)
    lead = lambda a: np.moveaxis(a, 0, 1)[None]  # noqa: E731  [n,H,d] -> [1,H,n,d]
    O, W = chunk_forward(lead(x["q"]), lead(x["k"]), lead(x["v"]), x["beta"].T[None], -1.0, 1, loss="mse", w0=x["s0"])
    assert np.allclose(np.moveaxis(O[0], 0, 1), o, rtol=1e-12, atol=1e-12) and np.allclose(W, final, rtol=1e-12, atol=1e-12)


def test_a_full_step_on_a_unit_key_stores_its_value(rng):
    x = _inputs(rng, 6, 1, 1, 5, 3, 1)
    big = np.full((6, 1), 60.0)   # eta = 1
    for n in range(1, 7):
        _, S = dr.forward(x["q"][:n], x["k"][:n], x["v"][:n], x["gate"][:n], big[:n], [0, n], "sigmoid", 1.0, x["s0"])
        assert np.allclose(S[0, 0].T @ x["k"][n - 1, 0], x["v"][n - 1, 0], atol=1e-12)


def test_sequences_are_independent_and_resume(rng):
    x = _inputs(rng, 20, 2, 1, 4, 3, 3)
    args = lambda a, b: [x[m][a:b] for m in ("q", "k", "v", "gate", "beta")]  # noqa: E731
    o, final = dr.forward(*args(0, 20), [0, 7, 7, 20], "sigmoid", 0.5, x["s0"])
    assert np.array_equal(final[1], x["s0"][1])
    part, mid = dr.forward(*args(7, 12), [0, 5], "sigmoid", 0.5, x["s0"][2:])
    rest, end = dr.forward(*args(12, 20), [0, 8], "sigmoid", 0.5, mid)
    assert np.allclose(np.concatenate([part, rest]), o[7:]) and np.allclose(end[0], final[2])


@pytest.mark.parametrize("kind", ["sigmoid", "log", None])
def test_backward_finite_differences(rng, kind):
    n, starts = 7, [0, 3, 3, 7]
    x = _inputs(rng, n, 4, 2, 3, 2, 3)
    x["gate"] = None if kind is None else -np.abs(x["gate"]) if kind == "log" else x["gate"]
    d_o, dsf = rng.standard_normal((n, 4, 2)), rng.standard_normal((3, 4, 3, 2))
    kw = dict(lr_max=1.5, lr_bias=0.3)

    def loss(y):
        o, f = dr.forward(y["q"], y["k"], y["v"], y["gate"], y["beta"], starts, kind, 0.7, y["s0"], **kw)
        return (o * d_o).sum() + (f * dsf).sum()

    g = dr.backward(x["q"], x["k"], x["v"], x["gate"], x["beta"], starts, kind, 0.7, d_o, x["s0"], dsf, **kw)
    for name in ("q", "k", "v", "gate", "beta", "s0"):
        if x[name] is None:
            continue
        for _ in range(6):
            at = tuple(rng.integers(0, s) for s in x[name].shape)
            up, down = ({**x, name: x[name].copy()} for _ in range(2))
            up[name][at] += 1e-5
            down[name][at] -= 1e-5
            want = (loss(up) - loss(down)) / 2e-5
            assert abs(g["d" + name][at] - want) <= 1e-7 * (1 + abs(want)), (name, at)


@pytest.mark.parametrize("pairing", ["half", "interleaved"])
def test_rotation_keeps_lengths_and_depends_on_distances_only(rng, pairing):
    freq = 10.0 ** -np.arange(3.0)
    x, y = rng.standard_normal((1, 1, 8)), rng.standard_normal((1, 1, 8))
    a = qk.turn(x, [11], freq, pairing)
    assert np.allclose(np.linalg.norm(a), np.linalg.norm(x)) and np.array_equal(a[..., 6:], x[..., 6:])
    assert np.allclose((a * qk.turn(y, [4], freq, pairing)).sum(), (qk.turn(x, [107], freq, pairing) * qk.turn(y, [100], freq, pairing)).sum())
    assert np.allclose(qk.turn(a, [11], freq, pairing, back=True), x)
    # a quarter turn of the first pair
    e = np.zeros((1, 1, 8))
    e[..., 0] = 1
    b = qk.turn(e, [1], [np.pi / 2] * 3, pairing)[0, 0]
    assert np.allclose(b, np.eye(8)[3 if pairing == "half" else 1])


@pytest.mark.parametrize("norm", ["none", "rms", "l2"])
def test_qknorm_backward_finite_differences(rng, norm):
    x, w, dy = rng.standard_normal((3, 2, 6)), rng.normal(1, 0.3, 6), rng.standard_normal((3, 2, 6))
    args = ([0, 5, -3], [1.0, 0.1], norm, "half")
    f = lambda x_, w_: (qk.forward(x_, w_, *args, eps=0.01, scale=1.3) * dy).sum()  # noqa: E731
    dx, dw = qk.backward(x, w, *args, dy, eps=0.01, scale=1.3)
    for at in np.ndindex(*x.shape):
        d = np.zeros_like(x)
        d[at] = 1e-5
        assert abs((f(x + d, w) - f(x - d, w)) / 2e-5 - dx[at]) < 1e-7
    for j in range(6):
        d = np.zeros(6)
        d[j] = 1e-5
        assert abs((f(x, w + d) - f(x, w - d)) / 2e-5 - dw[j]) < 1e-7
    h = qk.forward(x, None, [0] * 3, [], norm, "half", eps=0.0)
    size = {"none": None, "rms": np.sqrt(6.0), "l2": 1.0}[norm]
    assert np.allclose(h, x) if size is None else np.allclose(np.linalg.norm(h, axis=-1), size)
