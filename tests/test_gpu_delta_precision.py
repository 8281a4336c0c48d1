"""GPU tests of how exact the gated delta rule is in bf16: beside the rounding of an output there is what fp32 loses.

Errors are 2-norms over that of the fp64 result.  An output may be off by what the fp64 result is off when it is rounded
once (2^-8 of a value at most), and by what operands of two bf16 terms lose: 2^-17 of an operand, of at most four on
the way, in sums whose terms' magnitudes are together at most four times the result's: 2^-13.  What makes a state goes in
as three terms, but for T and the state itself: two, which lose 2^-18 / 3 in the root of squares (two roundings, each
uniform within half a step), so both of them sqrt(2) 2^-19.6, and fp32's own sums less than 2^-21: 2^-19.  In the
gate's gradient terms of another size than the result cancel: at most 16 times its size here, 2^-11; where there is
one token, its terms are taken as they are."""
import numpy as np
import pytest

from tests.block_utils import f64
from tests.test_gpu_delta import _make, _oracle, _train

pytestmark = pytest.mark.gpu

# sequences, tokens, heads, key heads, dk, dv: one chunk and many, narrow and wide, walks of two waves and of four
SHAPES = [(2, 7, 3, 3, 64, 64), (1, 64, 4, 4, 128, 128), (2, 300, 2, 1, 64, 64), (1, 300, 2, 2, 128, 96), (3, 200, 2, 2, 16, 16),
          (70, 130, 4, 2, 32, 64), (1, 150, 2, 2, 256, 64), (1, 2700, 1, 1, 64, 64)]


def _norm(x):
    return float(np.linalg.norm(x))


def _once(ref):
    """What rounding the fp64 result to bf16 loses."""
    import torch
    return _norm(f64(torch.from_numpy(ref.astype(np.float32)).to(torch.bfloat16)) - ref) / _norm(ref)


@pytest.mark.parametrize("j", range(len(SHAPES)))
def test_bf16_results_are_fp32_s_rounded_once(j):
    Bn, T, H, Hk, dk, dv = SHAPES[j]
    kind = ["sigmoid", "log"][j % 2]
    inp = _make(200 + j, Bn * T, Bn, H, Hk, dk, dv, "bf16", kind)
    inp["s0"] *= 0.3
    inp["d_sf"] *= 0.3
    out, want = _train(inp, kind, "bf16", B_=Bn, T=T), _oracle(inp, list(range(0, Bn * T + 1, T)), kind, dk ** -0.5)
    errs = {m: (_norm(f64(out[m]) - want[m]) / _norm(want[m]), _once(want[m])) for m in want if m not in ("s_final", "ds0")}
    states = {m: _norm(f64(out[m]) - want[m]) / _norm(want[m]) for m in ("s_final", "ds0")}
    print(f"[delta] {SHAPES[j]} " + " ".join(f"{m}={e:.1e}" for m, e in states.items()) + " " + " ".join(f"{m}={e:.2e}/{r:.2e}" for m, (e, r) in errs.items()), flush=True)
    assert all(e <= r + (2.0 ** -11 if m == "dgate" else 2.0 ** -13) for m, (e, r) in errs.items()), errs
    assert all(e <= 2.0 ** -19 for e in states.values()), states


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 32), (16, 16)])
@pytest.mark.parametrize("kind", ["sigmoid", "log"])
def test_the_gate_s_gradient_of_one_token(dk, dv, kind):
    """da = <dS', S> and terms of the token's own, each of which may be far larger than their sum: two bf16 terms of both
    operands lose 2^-16 of each product at most."""
    for seed in range(6):
        inp = _make(300 + seed, 1, 1, 1, 1, dk, dv, "bf16", kind)
        inp["s0"] *= 0.3
        inp["d_sf"] *= 0.3
        out, want = _train(inp, kind, "bf16", B_=1, T=1), _oracle(inp, [0, 1], kind, dk ** -0.5)
        x = {m: np.abs(f64(v)) for m, v in inp.items()}
        grow = x["d_sf"][0, 0] + dk ** -0.5 * np.outer(x["q"][0, 0], x["d_o"][0, 0])   # the state's gradient, by magnitudes
        terms = (x["s0"][0, 0] * grow).sum() + np.outer(x["k"][0, 0], x["k"][0, 0] @ grow).ravel() @ x["s0"][0, 0].ravel()
        err = abs(float(f64(out["dgate"])[0, 0]) - want["dgate"][0, 0])
        print(f"[delta] {kind} {dk} x {dv}: {want['dgate'][0, 0]:.2e} off by {err:.1e}, terms {terms:.1e}", flush=True)
        slope = 1.0 if kind == "log" else float(1 / (1 + np.exp(f64(inp["gate"])[0, 0])))
        assert err <= 2.0 ** -8 * abs(want["dgate"][0, 0]) + 2.0 ** -16 * slope * terms, (err, terms)
        err = abs(float(f64(out["dbeta"])[0, 0]) - want["dbeta"][0, 0])
        toward = x["k"][0, 0] @ grow
        parts = (toward * (x["v"][0, 0] + x["k"][0, 0] @ x["s0"][0, 0])).sum()
        assert err <= 2.0 ** -8 * abs(want["dbeta"][0, 0]) + 2.0 ** -16 * parts, (err, parts)
