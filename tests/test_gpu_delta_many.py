"""GPU tests of the gated delta rule where many heads' walks fill the chip (four chain waves a workgroup, chunks in turn
through two LDS buffers), and where few heads' long sequences are walked in pieces, against the fp64 token loop.
Tolerances are those of test_gpu_delta."""
import numpy as np
import pytest

from chunkwise_weight_recurrence_amd import binding as B
from tests.block_utils import f64
from tests.test_gpu_delta import CHUNK_TOL, _check, _make, _oracle, _train

pytestmark = pytest.mark.gpu


def _repeated(inp, lengths, times):
    """The sequences `lengths` of `inp`, `times` times one behind the other."""
    n = sum(lengths)
    return {k: v.repeat(times, *[1] * (v.dim() - 1)) for k, v in inp.items() if v.shape[0] in (n, len(lengths))}


def _forward_only(inp, kind, dtype, starts, B_, T):
    """o and s_final of a forward that keeps nothing for a backward."""
    import torch
    x = {k: v.cuda() for k, v in inp.items()}
    n, Hk, dk = inp["q"].shape
    H, dv = inp["v"].shape[1:]
    desc = B.make_delta_desc(B_, n if starts else T, H, dk, dv, Hk=Hk, dtype=dtype, gate=kind, packed=bool(starts))
    ws = torch.full((B.ttt_delta_workspace_size(desc, B.ENTRY_FWD),), 255, dtype=torch.uint8, device="cuda")
    out = dict(o=torch.full_like(x["v"], float("nan")), s_final=torch.full_like(x["s0"], float("nan")))
    B.ttt_delta_fwd(desc, x["q"], x["k"], x["v"], x["gate"], x["beta"], x["s0"], torch.tensor(starts, dtype=torch.int32).cuda() if starts else None,
                    out["o"], out["s_final"], None, ws)
    torch.cuda.synchronize()
    return out


# heads, key heads, dk, dv; rounds of the five sequences.  Every one is wide enough for four waves: sequences x heads x
# ceil(dv / 64) of at least 256.  Five sequences in turn, so that no two on one XCD or CU have to be the same.
MANY = [(4, 4, 128, 128, 7), (6, 2, 128, 100, 5), (4, 2, 70, 72, 7), (8, 8, 64, 64, 7), (6, 3, 50, 40, 9), (4, 1, 96, 250, 4)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("packed", [False, True])
def test_many_heads(dtype, packed):
    for j, (H, Hk, dk, dv, times) in enumerate(MANY):
        lengths = [200, 131, 64, 277, 1] if packed else [215] * 5
        kind = ["sigmoid", "log"][j % 2]
        n, S = sum(lengths), len(lengths) * times
        assert S * H * -(-dv // 64) >= 256   # the bound of four waves
        one = _make(100 + j, n, 5, H, Hk, dk, dv, dtype, kind)
        inp = _repeated(one, lengths, times)
        starts = np.concatenate([[0], np.cumsum(lengths * times)]).tolist()
        want = _oracle(one, starts[:6], kind, dk ** -0.5)
        out = _train(inp, kind, dtype, starts=starts if packed else None, B_=S, T=lengths[0])
        alone = _forward_only(inp, kind, dtype, starts if packed else None, S, lengths[0])
        for r in range(times):
            part = {m: v[r * (5 if m in ("s_final", "ds0") else n):][:5 if m in ("s_final", "ds0") else n] for m, v in out.items()}
            if r == 0:
                _check(part, want, dtype, what=f"{dtype} many {packed} {MANY[j]}")
                _check({m: v[:5 if m == "s_final" else n] for m, v in alone.items()}, {m: want[m] for m in alone}, dtype,
                       what=f"{dtype} forward alone")
                first, first_alone = part, alone
            else:   # the same sequences give the same bits wherever they lie
                for m in part:
                    assert np.array_equal(f64(part[m]), f64(first[m])), (m, r)
                for m, k in (("o", n), ("s_final", 5)):
                    assert np.array_equal(f64(alone[m][r * k:(r + 1) * k]), f64(first_alone[m][:k])), (m, r)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,dk,dv,chunks,tail", [(1, 256, 32, 60, 5), (1, 200, 96, 64, 9), (3, 64, 64, 48, 0), (1, 128, 128, 72, 31)])
def test_pieces_are_walked_and_joined(dtype, H, dk, dv, chunks, tail):
    """Slow decays, so that what enters a piece still counts when it leaves.  A token keeps e^-0.0025 on average, a chunk
    0.86 (bf16) or 0.92: a state's error a chunk, CHUNK_TOL in bf16 and three sums of 128 terms in fp32, adds up to 7 or
    13 of it, once more for the maps, and twice that for sums of 256 terms.  bf16 outputs and gradients as elsewhere."""
    C = 64 if dtype == "bf16" else 32
    T = chunks * C + tail
    inp = _make(chunks, T, 1, H, 1, dk, dv, dtype, "log")
    inp["gate"] = inp["gate"] * (1.0 / 64)   # the mean of |N(3, 1.5)| is 3.05: 3.05 x 0.05 / 64 a token
    inp["s0"] *= 0.3
    B.ttt_timing_enable(True)
    try:
        out = _train(inp, "log", dtype, B_=1, T=T)
        launches = B.ttt_timing_read(B.Kernel.DELTA_MAP)[1]
    finally:
        B.ttt_timing_enable(False)
    assert launches > 0, "the forward was not walked in pieces"
    state_tol = 2 * 2 * 7 * CHUNK_TOL if dtype == "bf16" else 2 * 2 * 13 * 3 * 128 * 2.0 ** -24
    _check(out, _oracle(inp, [0, T], "log", dk ** -0.5), dtype, state_tol=state_tol, tol=state_tol if dtype == "f32" else None,
           what=f"{dtype} pieces {H} x {dk} x {dv}")
