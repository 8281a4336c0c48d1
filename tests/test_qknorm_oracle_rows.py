"""The query and key norm's oracle, a row at a time (CPU)."""
import numpy as np
import pytest

from oracle import qknorm_oracle as qk


@pytest.mark.parametrize("norm", ["rms", "l2"])
def test_a_row_of_zeros_without_eps_changes_no_other(norm):
    """0 / 0 in its own row, as the formula has it, and the other rows' norms as they are alone."""
    rng = np.random.default_rng(0)
    x, dy = rng.standard_normal((5, 2, 6)), rng.standard_normal((5, 2, 6))
    x[3, 1] = 0
    pos, freq = np.arange(5), np.array([1.0, 0.1])
    y = qk.forward(x, None, pos, freq, norm, "half", eps=0.0)
    dx, _ = qk.backward(x, None, pos, freq, norm, "half", dy, eps=0.0)
    for t in range(5):
        for h in range(2):
            if (t, h) == (3, 1):
                assert np.isnan(y[t, h]).all() and np.isnan(dx[t, h]).all()
                continue
            size = np.sqrt((x[t, h] ** 2).mean() if norm == "rms" else (x[t, h] ** 2).sum())
            assert np.allclose(y[t, h], qk.turn((x[t, h] / size)[None, None], pos[t:t + 1], freq, "half")[0, 0], rtol=1e-13, atol=0)
            one = qk.backward(x[t:t + 1, h:h + 1], None, pos[t:t + 1], freq, norm, "half", dy[t:t + 1, h:h + 1], eps=0.0)[0]
            assert np.allclose(dx[t, h], one[0, 0], rtol=1e-12, atol=1e-14) and np.isfinite(one).all()
