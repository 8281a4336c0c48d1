"""GPU tests of the query and key norm at the ends of its rows and its turned columns: widths that are an odd number of
16-byte pieces, after other work has left NaN in LDS, and infinities where nothing is turned.  Tolerances are those of test_gpu_qknorm."""
import pytest

from chunkwise_weight_recurrence_amd import binding as B
from tests.test_gpu_qknorm import _check, _make, _run

pytestmark = pytest.mark.gpu


def _leave_in_lds(value):
    """A backward whose workgroups leave ``value`` in 16 KB of LDS each, in eight of them on every CU."""
    import torch
    n, H, d = 4096, 4, 512
    x = torch.ones(n, H, d, dtype=torch.bfloat16, device="cuda")
    dy = torch.full_like(x, value)
    dw = torch.empty(d, device="cuda")
    desc = B.make_qknorm_desc(n, H, 0, d, rot=0, norm="none")
    ws = torch.empty(B.ttt_qknorm_workspace_size(desc), dtype=torch.uint8, device="cuda")
    B.ttt_qknorm_bwd(desc, x, None, None, None, None, None, dy, None, torch.empty_like(x), None, dw, None, ws)
    torch.cuda.synchronize()
    assert torch.isnan(dw).all() if value != value else (dw == value * n * H).all()


@pytest.mark.parametrize("dtype,d,rot", [("bf16", 8, 8), ("bf16", 24, 24), ("bf16", 40, 16), ("bf16", 136, 136), ("f32", 12, 12), ("f32", 100, 40)])
@pytest.mark.parametrize("norm", ["rms", "l2", "none"])
def test_rows_that_end_in_half_a_unit(dtype, d, rot, norm):
    """Interleaved pairs: what earlier work left in LDS reaches no row.  One token a workgroup, and several with a rest."""
    import torch
    for n in (5, 1500, 4099):
        inp = _make(d + n, n, 3, 2, d, rot, dtype, True, False)
        outs = []
        for value in (0.0, float("nan")):
            _leave_in_lds(value)
            outs.append(_run(inp, dtype, norm, "interleaved", 1e-6, 1.0))
        print(f"[qknorm] {dtype} {norm} {n} x {d}", flush=True)
        for m in outs[0]:
            assert torch.equal(outs[0][m], outs[1][m]), m
        _check(inp, outs[1], dtype, norm, "interleaved", 1e-6, 1.0)


@pytest.mark.parametrize("dtype,d,rot", [("bf16", 64, 32), ("bf16", 64, 0), ("bf16", 40, 4), ("bf16", 70, 34), ("f32", 12, 2), ("f32", 33, 6)])
@pytest.mark.parametrize("pairing", ["half", "interleaved"])
def test_columns_that_are_not_turned_do_not_meet(dtype, d, rot, pairing):
    """An infinity or NaN behind the turned columns stays in its own, in both directions."""
    import torch
    inp = _make(d, 6, 2, 1, d, rot, dtype, True, False)
    clean = _run(inp, dtype, "none", pairing, 1e-6, 1.0)
    for bad in (float("inf"), float("nan")):
        for c in sorted({rot, rot + 1, d - 2, d - 1}):
            for x, m in (("q", "yq"), ("dyq", "dq")):
                dirty = {**inp, x: inp[x].clone()}
                dirty[x][3, 1, c] = bad
                got = _run(dirty, dtype, "none", pairing, 1e-6, 1.0)[m]
                assert not torch.isfinite(got[3, 1, c]) and torch.isnan(got[3, 1, c]).item() == (bad != bad), (m, bad, c)
                want = clean[m].clone()
                want[3, 1, c] = got[3, 1, c] = 0
                assert (got == want).all(), (m, bad, c)
    # a row with an infinity has the norm's factor 0: the other columns are zero
    dirty = {**inp, "q": inp["q"].clone()}
    dirty["q"][3, 1, d - 1] = float("inf")
    y = _run(dirty, dtype, "rms", pairing, 1e-6, 1.0)["yq"][3, 1]
    assert torch.isnan(y[d - 1]) and (y[:d - 1] == 0).all()


@pytest.mark.parametrize("dtype,d,rot", [("bf16", 64, 32), ("bf16", 70, 34), ("f32", 64, 64), ("f32", 33, 6)])
def test_without_a_norm_the_gradient_does_not_know_the_values(dtype, d, rot):
    import torch
    inp = _make(d, 6, 2, 1, d, rot, dtype, True, False)
    clean = _run(inp, dtype, "none", "half", 1e-6, 1.0)
    for bad in (float("inf"), float("nan")):
        dirty = {**inp, "q": inp["q"].clone()}
        dirty["q"][3, 1, 2] = dirty["q"][4, 0, d - 1] = bad
        assert (_run(dirty, dtype, "none", "half", 1e-6, 1.0)["dq"] == clean["dq"]).all(), bad


@pytest.mark.parametrize("norm", ["rms", "l2"])
def test_a_row_of_zeros_without_eps(norm):
    """0 / 0 in its own row; the others as the oracle has them."""
    import torch
    inp = _make(2, 9, 3, 2, 64, 32, "f32", False, False)
    keep = torch.ones(9, 3, dtype=torch.bool)
    keep[4, 1] = False
    inp["q"][4, 1] = 0
    out = _run(inp, "f32", norm, "half", 0.0, 1.0)
    assert torch.isnan(out["yq"][4, 1]).all() and torch.isnan(out["dq"][4, 1]).all() and torch.isnan(out["dwq"]).all()
    # the same rows without that one
    rest = {**inp, "q": inp["q"][keep][:, None], "dyq": inp["dyq"][keep][:, None], "k": torch.ones(26, 1, 64), "dyk": torch.ones(26, 1, 64),
            "pos": inp["pos"][:, None].expand(9, 3)[keep].contiguous()}
    got = dict(yq=out["yq"].cpu()[keep], dq=out["dq"].cpu()[keep])
    alone = _run(rest, "f32", norm, "half", 0.0, 1.0)
    _check(rest, alone, "f32", norm, "half", 0.0, 1.0)
    for m in got:
        assert torch.equal(got[m], alone[m].cpu()[:, 0]), m
