"""GPU tests of the query and key norm at the ends of its rows: widths that are an odd number of 16-byte pieces, after
other work has left NaN in LDS.  Tolerances are those of test_gpu_qknorm."""
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
