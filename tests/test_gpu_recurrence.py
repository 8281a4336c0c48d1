"""GPU tests of the gated linear recurrence against the fp64 token loops, at every
place where the token axis is cut (128-token runs, sequence borders).

Tolerances: the oracle's running bound on fp32 arithmetic plus half a step of the
output's type (``tests/block_utils.py::worst``; above 1 is wrong)."""
import numpy as np
import pytest

from chunkwise_weight_recurrence_amd import binding as B
from oracle import recurrence_oracle as rec
from tests.block_utils import HALF, f64, rounded, torch_dtype, worst

pytestmark = pytest.mark.gpu


def _make(seed, n, S, D, dtype, gate, z_mean=3.0):
    rng = np.random.default_rng(seed)
    x = rounded(rng, (n, D), dtype)
    z = rounded(rng, (n, D), dtype, mean=z_mean, std=1.5)
    if gate == "log":
        z = -(z.float().abs() * 0.05).to(z.dtype)
    return dict(x=x, z=z, h0=rounded(rng, (S, D), "f32"), d_o=rounded(rng, (n, D), dtype),
                d_hf=rounded(rng, (S, D), "f32"))


def _train(inp, gate, kind, dtype, starts=None, B_=None, T=None, states=True, poison=True):
    """Forward and backward on the GPU; packed with ``starts``, else dense [B_, T]."""
    import torch
    n, D = inp["x"].shape
    dev = {k: v.cuda() for k, v in inp.items()}
    packed = starts is not None
    desc = B.make_rec_desc(len(starts) - 1 if packed else B_, n if packed else T, D, dtype=dtype, gate=gate, input=kind,
                           packed=packed)
    st = torch.tensor(starts, dtype=torch.int32).cuda() if packed else None
    io = dict(dtype=torch_dtype(dtype), device="cuda")
    f32 = dict(dtype=torch.float32, device="cuda")
    S = desc.B
    fill = float("nan") if poison else 0.0
    out = dict(o=torch.full((n, D), fill, **io), h_final=torch.full((S, D), fill, **f32), dx=torch.full((n, D), fill, **io),
               dgate=torch.full((n, D), fill, **io), dh0=torch.full((S, D), fill, **f32))
    size = max(B.ttt_recurrence_workspace_size(desc, e) for e in (0, 1))
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda") if size else None
    saved = torch.full((B.ttt_recurrence_saved_size(desc),), 255, dtype=torch.uint8, device="cuda")
    h0 = dev["h0"] if states else None
    B.ttt_recurrence_fwd(desc, dev["x"], dev["z"], h0, st, out["o"], out["h_final"] if states else None, saved, ws)
    B.ttt_recurrence_bwd(desc, dev["x"], dev["z"], h0, st, saved, dev["d_o"], dev["d_hf"] if states else None, out["dx"],
                         out["dgate"], out["dh0"] if states else None, ws)
    torch.cuda.synchronize()
    return out


def _check(inp, out, starts, gate, kind, dtype, states=True):
    x, z, d_o = (f64(inp[k]) for k in ("x", "z", "d_o"))
    h0, dhf = (f64(inp["h0"]), f64(inp["d_hf"])) if states else (None, None)
    o, hf, eo, ef = rec.forward(x, z, starts, gate, kind, h0)
    g = rec.backward(x, z, starts, gate, kind, d_o, h0, dhf)
    errs = dict(o=worst(out["o"], o, eo, dtype), dx=worst(out["dx"], g["dx"], g["e_dx"], dtype),
                dgate=worst(out["dgate"], g["dgate"], g["e_dgate"], dtype))
    if states:
        errs.update(h_final=worst(out["h_final"], hf, ef, "f32"), dh0=worst(out["dh0"], g["dh0"], g["e_dh0"], "f32"))
    assert all(e <= 1.0 for e in errs.values()), errs


KINDS = [("sigmoid", "convex"), ("sigmoid", "plain"), ("log", "convex"), ("log", "plain")]
DENSE = [(1, 1, 1), (1, 1, 3), (3, 5, 65), (2, 16, 64), (2, 17, 130), (1, 127, 128), (1, 128, 8), (2, 129, 96),
         (1, 257, 200), (5, 60, 7), (2, 700, 2), (70, 3, 10), (200, 1, 66)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate,kind", KINDS)
def test_dense(dtype, gate, kind):
    for k, (Bn, T, D) in enumerate(DENSE):
        inp = _make(k, Bn * T, Bn, D, dtype, gate)
        states = k % 3 != 2
        out = _train(inp, gate, kind, dtype, B_=Bn, T=T, states=states)
        _check(inp, out, rec.dense_starts(Bn, T), gate, kind, dtype, states)


LENGTHS = [[1], [128], [129], [0, 0, 5, 0], [127, 1, 128, 129, 0, 300], [16] * 20, [1] * 150, [0] * 90 + [3] + [0] * 90,
           [1000], [5, 900, 0, 0, 1, 1, 200], [0] * 5000 + [7, 250]]


@pytest.mark.parametrize("dtype,D", [("bf16", 70), ("bf16", 33), ("f32", 65)])
@pytest.mark.parametrize("gate,kind", [("sigmoid", "convex"), ("log", "plain")])
def test_packed(dtype, D, gate, kind):
    for k, lens in enumerate(LENGTHS):
        starts = np.concatenate([[0], np.cumsum(lens)]).tolist()
        inp = _make(100 + k, starts[-1], len(lens), D, dtype, gate)
        out = _train(inp, gate, kind, dtype, starts=starts, states=k % 2 == 0)
        _check(inp, out, starts, gate, kind, dtype, states=k % 2 == 0)


def test_no_tokens_passes_the_states_on():
    import torch
    for starts, T in (([0, 0, 0], None), (None, 0)):
        inp = _make(1, 0, 2, 40, "bf16", "sigmoid")
        out = _train(inp, "sigmoid", "convex", "bf16", starts=starts, B_=2, T=T)
        assert torch.equal(out["h_final"].cpu(), inp["h0"]) and torch.equal(out["dh0"].cpu(), inp["d_hf"])


def test_rows_outside_the_sequences_are_left_alone():
    import torch
    starts, n, D = [7, 140, 140, 301], 600, 48
    inp = _make(5, n, 3, D, "bf16", "sigmoid")
    outside = torch.ones(n, dtype=torch.bool)
    outside[7:301] = False
    for k in ("x", "z", "d_o"):
        inp[k][outside] = float("nan")
    out = _train(inp, "sigmoid", "convex", "bf16", starts=starts)
    for k in ("o", "dx", "dgate"):
        assert torch.isnan(out[k].cpu()[outside]).all()   # as they were: the buffers start as NaN
        assert not torch.isnan(out[k].cpu()[~outside]).any()
    same = {k: v if k in ("h0", "d_hf") else v[7:301] for k, v in inp.items()}
    _check(same, {k: v if k in ("h_final", "dh0") else v[7:301] for k, v in out.items()}, [0, 133, 133, 294], "sigmoid",
           "convex", "bf16")
    out = _train(inp, "sigmoid", "convex", "bf16", starts=starts, poison=False)
    for k in ("o", "dx", "dgate"):
        assert (out[k].cpu()[outside] == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_values_stay_in_their_sequence(bad):
    import torch
    lens = [130, 50, 200, 3, 260]
    starts = np.concatenate([[0], np.cumsum(lens)]).tolist()
    clean = _make(6, starts[-1], 5, 64, "bf16", "sigmoid")
    dirty = {k: v.clone() for k, v in clean.items()}
    for s in (1, 3):
        for k in ("x", "z", "d_o"):
            dirty[k][starts[s]:starts[s + 1]] = bad
        dirty["h0"][s] = bad
        dirty["d_hf"][s] = bad
    a, b = (_train(i, "sigmoid", "convex", "bf16", starts=starts) for i in (clean, dirty))
    for s in (0, 2, 4):
        for k in ("o", "dx", "dgate"):
            assert torch.equal(a[k][starts[s]:starts[s + 1]], b[k][starts[s]:starts[s + 1]])
        for k in ("h_final", "dh0"):
            assert torch.equal(a[k][s], b[k][s])
    # and a NaN reaches every later token of its own
    one = {k: v.clone() for k, v in clean.items()}
    one["x"][starts[4] + 2] = float("nan")
    c = _train(one, "sigmoid", "convex", "bf16", starts=starts)
    assert torch.isnan(c["o"][starts[4] + 2:]).all() and torch.isnan(c["h_final"][4]).all()
    assert torch.equal(c["o"][:starts[4] + 2], a["o"][:starts[4] + 2])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extreme_gates(dtype):
    """Gates that forget everything, keep everything, or lie far out on either side."""
    n, D = 300, 64
    for gate, values in (("sigmoid", [-float("inf"), float("inf"), -90.0, 90.0, -30.0, 0.0]),
                         ("log", [-float("inf"), 0.0, -100.0, -1e-6, -0.5, -0.51])):
        for kind in ("convex", "plain"):
            inp = _make(7, n, 1, D, dtype, gate)
            inp["x"] *= 0.1
            for k, v in enumerate(values):
                inp["z"][k * 50:k * 50 + 3] = v
                inp["z"][k * 50 + 20, ::2] = v
            out = _train(inp, gate, kind, dtype, starts=[0, n])
            _check(inp, out, [0, n], gate, kind, dtype)


def test_keep_everything_is_a_running_sum():
    n, D = 1500, 8
    inp = _make(8, n, 1, D, "f32", "log")
    inp["z"].zero_()
    out = _train(inp, "log", "plain", "f32", starts=[0, n])
    _check(inp, out, [0, n], "log", "plain", "f32")


def test_strided_rows():
    """x and gate as two halves of one projection, their gradients into two halves of another."""
    import torch
    from chunkwise_weight_recurrence_amd.layer import RecurrenceBuffers
    for Bn, T, D, pad in ((2, 150, 64, 0), (1, 300, 33, 0), (3, 140, 66, 1)):
        inp = _make(9, Bn * T, Bn, D, "bf16", "sigmoid")
        # the second half starts on a 16-byte boundary, rows are D + room (+ pad) elements apart
        room = -(-D // 8) * 8
        both = torch.full((Bn, T, 2 * room + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
        x, z = both[..., :D], both[..., room:room + D]
        x.copy_(inp["x"].view(Bn, T, D))
        z.copy_(inp["z"].view(Bn, T, D))
        buf = RecurrenceBuffers(x, z, h0=inp["h0"].cuda(), with_bwd=True)
        dboth = torch.full_like(both, 7.0)
        buf.dx, buf.dgate = dboth[..., :D], dboth[..., room:room + D]
        buf.forward()
        buf.backward(inp["d_o"].view(Bn, T, D).cuda(), inp["d_hf"].cuda())
        torch.cuda.synchronize()
        out = dict(o=buf.o, h_final=buf.h_final, dh0=buf.dh0, dx=buf.dx.reshape(-1, D), dgate=buf.dgate.reshape(-1, D))
        _check(inp, out, rec.dense_starts(Bn, T), "sigmoid", "convex", "bf16")
        gaps = torch.ones(both.shape[-1], dtype=torch.bool)
        gaps[:D] = gaps[room:room + D] = False
        assert (dboth[..., gaps.cuda()] == 7.0).all()


def test_dense_and_packed_agree_and_repeat_to_the_bit():
    import torch
    Bn, T, D = 3, 333, 200
    inp = _make(10, Bn * T, Bn, D, "bf16", "sigmoid")
    a = _train(inp, "sigmoid", "convex", "bf16", B_=Bn, T=T)
    for _ in range(3):
        for b in (_train(inp, "sigmoid", "convex", "bf16", B_=Bn, T=T),
                  _train(inp, "sigmoid", "convex", "bf16", starts=rec.dense_starts(Bn, T).tolist())):
            assert all(torch.equal(a[k], b[k]) for k in a)


def test_long_sequences_and_resuming():
    """Many runs of tokens (also more than one group of runs), and the same in two parts through h_final and h0."""
    import torch
    n, D = 9000, 16
    inp = _make(11, n, 1, D, "f32", "sigmoid", z_mean=5.0)
    out = _train(inp, "sigmoid", "convex", "f32", starts=[0, n])
    _check(inp, out, [0, n], "sigmoid", "convex", "f32")
    cut = 4321
    first = {k: v if k in ("h0", "d_hf") else v[:cut] for k, v in inp.items()}
    a = _train(first, "sigmoid", "convex", "f32", starts=[0, cut])
    rest = {k: v if k in ("h0", "d_hf") else v[cut:].contiguous() for k, v in inp.items()}
    rest["h0"] = a["h_final"].cpu()
    b = _train(rest, "sigmoid", "convex", "f32", starts=[0, n - cut])
    x, z = f64(inp["x"]), f64(inp["z"])
    o, hf, eo, ef = rec.forward(x, z, [0, n], "sigmoid", "convex", f64(inp["h0"]))
    assert worst(torch.cat([a["o"], b["o"]]), o, eo, "f32") <= 1 and worst(b["h_final"], hf, ef, "f32") <= 1
    # the gradient that the second part hands back is what the first part's final state gets
    first["d_hf"] = b["dh0"].cpu()
    g = _train(first, "sigmoid", "convex", "f32", starts=[0, cut])
    want = rec.backward(x, z, [0, n], "sigmoid", "convex", f64(inp["d_o"]), f64(inp["h0"]), f64(inp["d_hf"]))
    assert worst(torch.cat([g["dx"], b["dx"]]), want["dx"], want["e_dx"], "f32") <= 1
    assert worst(g["dh0"], want["dh0"], want["e_dh0"], "f32") <= 1


@pytest.mark.parametrize("dtype,n,D,gate,kind", [("bf16", 4300, 16384, "sigmoid", "convex"), ("bf16", 4200, 16385, "log", "convex"),
                                                 ("f32", 9000, 8000, "sigmoid", "plain")])
def test_large_problems(dtype, n, D, gate, kind):
    """Enough tiles for the forward's larger ones, and for more than a group of them; checked on some channels."""
    lens = [n - 2911, 0, 1, 255, 256, 257, 2142]
    starts = np.concatenate([[0], np.cumsum(lens)]).tolist()
    assert starts[-1] == n
    for st in (starts, [0, n]):
        inp = _make(50, n, len(st) - 1, D, dtype, gate, z_mean=5.0)
        out = _train(inp, gate, kind, dtype, starts=st)
        at = np.unique(np.concatenate([[0, 1, 126, 127, 128, D - 130, D - 2, D - 1], np.random.default_rng(0).integers(0, D, 30)]))
        some = {k: v[:, at] for k, v in inp.items()}
        _check(some, {k: v[:, at] for k, v in out.items()}, st, gate, kind, dtype)


def test_one_tile_of_very_many_channels():
    inp = _make(51, 200, 2, 270_000, "bf16", "sigmoid")
    out = _train(inp, "sigmoid", "convex", "bf16", starts=[0, 70, 200])
    at = np.array([0, 1, 135_000, 269_998, 269_999])
    _check({k: v[:, at] for k, v in inp.items()}, {k: v[:, at] for k, v in out.items()}, [0, 70, 200], "sigmoid", "convex", "bf16")


def test_offsets_past_32_bits():
    """The last of two sequences lies behind the first 2^31 elements."""
    import torch
    n, D, tail = 140_000, 16_384, 200
    inp = _make(12, tail, 1, D, "bf16", "sigmoid")
    x = torch.zeros((n, D), dtype=torch.bfloat16, device="cuda")
    z = torch.zeros_like(x)
    x[-tail:], z[-tail:] = inp["x"].cuda(), inp["z"].cuda()
    o = torch.empty_like(x)
    starts = torch.tensor([0, n - tail, n], dtype=torch.int32).cuda()
    desc = B.make_rec_desc(2, n, D, packed=True)
    h0 = torch.cat([torch.zeros_like(inp["h0"]), inp["h0"]]).cuda()
    hf = torch.empty_like(h0)
    ws = torch.empty(B.ttt_recurrence_workspace_size(desc, 1), dtype=torch.uint8, device="cuda")
    saved = torch.empty(B.ttt_recurrence_saved_size(desc), dtype=torch.uint8, device="cuda")
    B.ttt_recurrence_fwd(desc, x, z, h0, starts, o, hf, saved, ws)
    want, whf, eo, ef = rec.forward(f64(inp["x"]), f64(inp["z"]), [0, tail], "sigmoid", "convex", f64(inp["h0"]))
    assert worst(o[-tail:], want, eo, "bf16") <= 1 and worst(hf[1:], whf, ef, "f32") <= 1
    assert not o[:n - tail].any() and not hf[0].any()
    d_o = torch.zeros_like(x)
    d_o[-tail:] = inp["d_o"].cuda()
    dz = torch.empty_like(x)
    dh0 = torch.empty_like(h0)
    # dx takes o's place, which is no longer needed
    B.ttt_recurrence_bwd(desc, x, z, h0, starts, saved, d_o, None, o, dz, dh0, ws)
    g = rec.backward(f64(inp["x"]), f64(inp["z"]), [0, tail], "sigmoid", "convex", f64(inp["d_o"]), f64(inp["h0"]))
    assert worst(o[-tail:], g["dx"], g["e_dx"], "bf16") <= 1 and worst(dz[-tail:], g["dgate"], g["e_dgate"], "bf16") <= 1
    assert worst(dh0[1:], g["dh0"], g["e_dh0"], "f32") <= 1
    assert not o[:n - tail].any() and not dz[:n - tail].any()


@pytest.mark.parametrize("dtype,D", [("bf16", 520), ("bf16", 37), ("f32", 300)])
@pytest.mark.parametrize("gate,kind", KINDS)
def test_step(dtype, D, gate, kind):
    import torch
    rows, pool = 9, 12
    inp = _make(13, rows, pool, D, dtype, gate)
    slots = [4, -1, 0, 11, 7, 12, 2, 9, 1]   # two rows of padding
    desc = B.make_rec_desc(rows, 1, D, dtype=dtype, gate=gate, input=kind)
    h = inp["h0"].cuda()
    o = torch.full((rows, D), 5.0, dtype=torch_dtype(dtype), device="cuda")
    B.ttt_recurrence_step(desc, inp["x"].cuda(), inp["z"].cuda(), torch.tensor(slots, dtype=torch.int32).cuda(), h, o)
    want_h, bound = f64(inp["h0"]), np.zeros((pool, D))
    for b, s in enumerate(slots):
        if not 0 <= s < pool:
            assert (o[b] == 5.0).all()
            continue
        w, hf, eo, ef = rec.forward(f64(inp["x"])[b:b + 1], f64(inp["z"])[b:b + 1], [0, 1], gate, kind, want_h[s:s + 1])
        want_h[s], bound[s] = hf[0], ef[0]
        assert worst(o[b], w[0], eo[0], dtype) <= 1
    assert worst(h, want_h, bound, "f32") <= 1
    untouched = [s for s in range(pool) if s not in slots]
    assert torch.equal(h[untouched].cpu(), inp["h0"][untouched])


def test_step_rows_of_one_slot_are_consecutive_tokens():
    """Also over more rows than a workgroup looks at together, and equal to the whole sequence at once."""
    import torch
    rows, D = 700, 24
    inp = _make(14, rows, 3, D, "f32", "sigmoid")
    rng = np.random.default_rng(3)
    slots = rng.choice([0, 1, 2, -1], size=rows, p=[0.5, 0.3, 0.1, 0.1])
    slots[0], slots[-1] = 2, 2
    h = inp["h0"].cuda()
    o = torch.full((rows, D), 5.0, device="cuda")
    desc = B.make_rec_desc(rows, 1, D, dtype="f32")
    B.ttt_recurrence_step(desc, inp["x"].cuda(), inp["z"].cuda(), torch.tensor(slots, dtype=torch.int32).cuda(), h, o)
    for s in range(3):
        at = np.flatnonzero(slots == s)
        w, hf, eo, ef = rec.forward(f64(inp["x"])[at], f64(inp["z"])[at], [0, len(at)], "sigmoid", "convex", f64(inp["h0"])[s:s + 1])
        assert worst(o[at.tolist()], w, eo, "f32") <= 1 and worst(h[s], hf[0], ef[0], "f32") <= 1
    assert (o[np.flatnonzero(slots < 0).tolist()] == 5.0).all()


def test_steps_continue_a_prompt():
    """Prefill, then single tokens from its final state: the same as the whole sequence."""
    import torch
    n, cut, D = 140, 131, 96
    inp = _make(15, 2 * n, 2, D, "bf16", "sigmoid")
    x, z = inp["x"].view(2, n, D).cuda(), inp["z"].view(2, n, D).cuda()
    o, h = torch.empty(2, cut, D, dtype=torch.bfloat16, device="cuda"), torch.empty(2, D, device="cuda")
    desc = B.make_rec_desc(2, cut, D)
    ws = torch.empty(B.ttt_recurrence_workspace_size(desc, 0), dtype=torch.uint8, device="cuda")
    B.ttt_recurrence_fwd(desc, x[:, :cut].contiguous(), z[:, :cut].contiguous(), inp["h0"].cuda(), None, o, h, None, ws)
    outs = [o]
    step = B.make_rec_desc(2, 1, D)
    for t in range(cut, n):
        o1 = torch.empty(2, 1, D, dtype=torch.bfloat16, device="cuda")
        B.ttt_recurrence_step(step, x[:, t].contiguous(), z[:, t].contiguous(), None, h, o1)
        outs.append(o1)
    want, hf, eo, ef = rec.forward(f64(inp["x"]), f64(inp["z"]), [0, n, 2 * n], "sigmoid", "convex", f64(inp["h0"]))
    assert worst(torch.cat(outs, 1).reshape(-1, D), want, eo, "bf16") <= 1 and worst(h, hf, ef, "f32") <= 1


def test_a_captured_step_reads_its_slots_at_each_replay():
    """A decode loop: one graph, with other rows, gates and slots for every token, against eager steps."""
    import torch
    rows, pool, D = 6, 9, 200
    inp = _make(16, 5 * rows, pool, D, "bf16", "sigmoid")
    desc = B.make_rec_desc(rows, 1, D)
    x, z = (inp[k].view(5, rows, D).cuda() for k in ("x", "z"))
    slots = torch.tensor([[0, 1, 2, 3, 4, 5], [5, 4, -1, 2, 1, 0], [8, 8, 8, 7, 0, 9], [-1] * 6, [6, 0, 6, 0, 6, 0]],
                         dtype=torch.int32).cuda()
    xs, zs, ss = torch.empty_like(x[0]), torch.empty_like(z[0]), torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    h, o = inp["h0"].cuda(), torch.zeros(rows, D, dtype=torch.bfloat16, device="cuda")
    he, oe = h.clone(), o.clone()
    B.ttt_recurrence_step(desc, xs, zs, ss, h, o)   # the library is loaded before the capture
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.ttt_recurrence_step(desc, xs, zs, ss, h, o)
    for t in range(5):
        xs.copy_(x[t])
        zs.copy_(z[t])
        ss.copy_(slots[t])
        g.replay()
        row = slots[t].clone()   # its own allocation: a pointer is 16-byte aligned
        B.ttt_recurrence_step(desc, x[t].clone(), z[t].clone(), row, he, oe)
        torch.cuda.synchronize()
        assert torch.equal(h, he) and torch.equal(o, oe), t


def test_two_graphs_share_a_workspace_and_replay():
    """Captured forwards and backwards of two problems over one workspace, replayed in turn
    with eager calls of both between them: every replay gives the eager results."""
    import torch
    from chunkwise_weight_recurrence_amd.layer import RecurrenceBuffers
    probs = []
    for k, (Bn, T, D) in enumerate(((2, 500, 128), (1, 900, 70))):
        inp = _make(20 + k, Bn * T, Bn, D, "bf16", "sigmoid")
        b = RecurrenceBuffers(inp["x"].view(Bn, T, D).cuda(), inp["z"].view(Bn, T, D).cuda(), h0=inp["h0"].cuda(), with_bwd=True)
        probs.append((b, inp["d_o"].view(Bn, T, D).cuda(), inp["d_hf"].cuda()))
    big = max((p[0].ws for p in probs), key=lambda w: w.numel())
    for p in probs:
        p[0].ws = big

    def both(p):
        p[0].forward()
        p[0].backward(p[1], p[2])

    def read(p):
        torch.cuda.synchronize()
        return [t.clone() for t in (p[0].o, p[0].h_final, p[0].dx, p[0].dgate, p[0].dh0)]

    eager = []
    for p in probs:
        both(p)
        eager.append(read(p))
    side = torch.cuda.Stream()
    graphs = []
    for p in probs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            both(p)
        graphs.append(g)
    for r in range(4):
        for k, p in enumerate(probs):
            for t in (p[0].o, p[0].h_final, p[0].dx, p[0].dgate, p[0].dh0):
                t.fill_(float("nan"))
            graphs[k].replay()
            assert all(torch.equal(a, b) for a, b in zip(read(p), eager[k])), (r, k)
            both(probs[1 - k])
            assert all(torch.equal(a, b) for a, b in zip(read(probs[1 - k]), eager[1 - k])), (r, k)


def test_two_streams_at_once():
    import torch
    from chunkwise_weight_recurrence_amd.layer import RecurrenceBuffers
    work = []
    for k in range(2):
        inp = _make(30 + k, 6000, 1, 512, "bf16", "sigmoid")
        b = RecurrenceBuffers(inp["x"].view(1, 6000, 512).cuda(), inp["z"].view(1, 6000, 512).cuda(), with_bwd=True)
        d_o = inp["d_o"].view(1, 6000, 512).cuda()
        b.forward()
        b.backward(d_o)
        torch.cuda.synchronize()
        work.append((b, d_o, [t.clone() for t in (b.o, b.dx, b.dgate, b.dh0)], torch.cuda.Stream()))
    for _ in range(20):
        for b, d_o, _, s in work:
            with torch.cuda.stream(s):
                b.forward()
                b.backward(d_o)
    torch.cuda.synchronize()
    for b, _, want, _ in work:
        assert all(torch.equal(a, c) for a, c in zip((b.o, b.dx, b.dgate, b.dh0), want))


def test_unsorted_starts_stay_inside_the_buffers():
    """Entries out of order or out of range give unspecified outputs, but end, and touch nothing else."""
    import torch
    n, D = 1000, 40
    for starts in ([0, 900, 100, 1000], [1000, 500, 0, 200], [-50, 2000, -7, 5000], [2 ** 31 - 1, -2 ** 31, 0, 3]):
        inp = _make(40, n, 3, D, "bf16", "sigmoid")
        _train(inp, "sigmoid", "convex", "bf16", starts=starts)


def test_single_strided_tokens():
    """[B,1,D] views of a projection: the rows' distance is that of the batch axis."""
    import torch
    from chunkwise_weight_recurrence_amd.layer import RecurrenceBuffers
    Bn, T, D = 5, 3, 48
    inp = _make(60, Bn, Bn, D, "bf16", "sigmoid")
    both = torch.full((Bn, T, 2 * D), float("nan"), dtype=torch.bfloat16, device="cuda")
    x, z = both[:, :1, :D], both[:, :1, D:]
    x.copy_(inp["x"].view(Bn, 1, D))
    z.copy_(inp["z"].view(Bn, 1, D))
    buf = RecurrenceBuffers(x, z, h0=inp["h0"].cuda(), with_bwd=True)
    dboth = torch.full_like(both, 7.0)
    buf.dx, buf.dgate = dboth[:, :1, :D], dboth[:, :1, D:]
    buf.forward()
    buf.backward(inp["d_o"].view(Bn, 1, D).cuda(), inp["d_hf"].cuda())
    out = dict(o=buf.o.view(Bn, D), h_final=buf.h_final, dh0=buf.dh0, dx=buf.dx.reshape(Bn, D), dgate=buf.dgate.reshape(Bn, D))
    _check(inp, out, rec.dense_starts(Bn, 1), "sigmoid", "convex", "bf16")
    assert (dboth[:, 1:] == 7.0).all()


def _exact_inputs(n, S, D, dtype, seed, halvings=8):
    """Inputs whose every state, gradient and map is exact in fp32 in whatever order it is formed: whole numbers as x
    and d_o, gates that keep everything (a = 1) but for a few tokens a channel where a is a half.  Made on the GPU."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def whole(*shape, dt=torch_dtype(dtype)):
        return torch.randint(-2, 3, shape, generator=gen, device="cuda").to(dt)

    z = torch.full((n, D), float("inf"), dtype=torch_dtype(dtype), device="cuda")
    z.scatter_(0, torch.randint(0, n, (halvings, D), generator=gen, device="cuda"), 0.0)
    return dict(x=whole(n, D), z=z, h0=whole(S, D, dt=torch.float32), d_o=whole(n, D), d_hf=whole(S, D, dt=torch.float32))


# Sequences over more than three groups of 32 tiles, so that maps of whole groups are read: a dense one, two of them, and
# packed ones whose long sequence begins and ends inside a group.  The last two have enough tiles for the forward's larger.
@pytest.mark.parametrize("dtype,D,starts", [
    ("bf16", 200, [0, 13000]), ("bf16", 201, [0, 13000]), ("f32", 130, [0, 13000]), ("f32", 67, [0, 13000, 26000]),
    ("bf16", 66, [0, 700, 25111, 25111, 26000]), ("bf16", 35, [300, 1000, 1001, 25000]),
    ("bf16", 2600, [0, 26000]), ("bf16", 2601, [0, 700, 25711, 26000]),
])
def test_a_long_way_back_is_exact(dtype, D, starts):
    """A map left out, read twice or in another place shows in every later token: nothing here is rounded but outputs."""
    import torch
    n, S = starts[-1], len(starts) - 1
    inp = _exact_inputs(n, S, D, dtype, seed=70)
    T = n // S
    runs = [dict(starts=starts)] + ([dict(B_=S, T=T)] if starts == list(range(0, n + 1, T)) else [])
    at = np.unique(np.linspace(0, D - 1, 40).astype(int))
    x, z, d_o, h0, dhf = (f64(inp[k][:, at]) for k in ("x", "z", "d_o", "h0", "d_hf"))
    o, hf, _, _ = rec.forward(x, z, starts, "sigmoid", "plain", h0)
    g = rec.backward(x, z, starts, "sigmoid", "plain", d_o, h0, dhf)
    assert max(np.abs(v).max() for v in (o, hf, g["dx"], g["dh0"])) < 2 ** 15   # 2^-8 .. 2^15: 23 bits
    for run in runs:
        out = {k: v[:, at] for k, v in _train(inp, "sigmoid", "plain", dtype, **run).items()}
        first = starts[0]
        for k, want, t in (("o", o, dtype), ("h_final", hf, "f32"), ("dx", g["dx"], dtype), ("dh0", g["dh0"], "f32")):
            want = torch.from_numpy(want).to(torch.float32).to(torch_dtype(t))
            got = out[k].cpu()
            if k in ("o", "dx"):
                want, got = want[first:], got[first:]
            assert torch.equal(got, want), (k, int((got != want).any(1).nonzero()[0]))
        # dgate is a quarter of dh h where the gate is a half, and zero elsewhere: a product, rounded
        assert worst(out["dgate"][first:], g["dgate"][first:], 2 * HALF["f32"] * np.abs(g["dgate"][first:]), dtype) <= 1


@pytest.mark.parametrize("D", [34, 33])
@pytest.mark.parametrize("gate,kind", KINDS)
def test_long_bf16_sequences(D, gate, kind):
    """More than three groups of tiles with ordinary gates, two channels a lane and one."""
    starts = [0, 300, 12900, 13000]
    inp = _make(71, 13000, 3, D, "bf16", gate, z_mean=5.0)
    _check(inp, _train(inp, gate, kind, "bf16", starts=starts), starts, gate, kind, "bf16")


def test_unsorted_starts_write_nothing_around_the_buffers():
    """Each output, the saved context and the workspace lies inside a larger buffer, whose rest stays as it was."""
    import torch
    n, D, S = 1000, 40, 3
    inp = {k: v.cuda() for k, v in _make(40, n, S, D, "bf16", "sigmoid").items()}
    desc = B.make_rec_desc(S, n, D, packed=True)
    sizes = dict(saved=B.ttt_recurrence_saved_size(desc), ws=max(B.ttt_recurrence_workspace_size(desc, e) for e in (0, 1)),
                 o=n * D * 2, dx=n * D * 2, dgate=n * D * 2, h_final=S * D * 4, dh0=S * D * 4)
    room = 1 << 16   # bytes on either side
    for starts in ([0, 900, 100, 1000], [1000, 500, 0, 200], [-50, 2000, -7, 5000], [2 ** 31 - 1, -2 ** 31, 0, 3], [0, 400, 1000, 700]):
        whole = {k: torch.full((size + 2 * room,), 0xA5, dtype=torch.uint8, device="cuda") for k, size in sizes.items()}
        part = {k: whole[k][room:room + size] for k, size in sizes.items()}
        for k in ("o", "dx", "dgate"):
            part[k] = part[k].view(torch.bfloat16).view(n, D)
        for k in ("h_final", "dh0"):
            part[k] = part[k].view(torch.float32).view(S, D)
        st = torch.tensor(starts, dtype=torch.int32).cuda()
        B.ttt_recurrence_fwd(desc, inp["x"], inp["z"], inp["h0"], st, part["o"], part["h_final"], part["saved"], part["ws"])
        B.ttt_recurrence_bwd(desc, inp["x"], inp["z"], inp["h0"], st, part["saved"], inp["d_o"], inp["d_hf"], part["dx"],
                             part["dgate"], part["dh0"], part["ws"])
        torch.cuda.synchronize()
        for k, size in sizes.items():
            assert (whole[k][:room] == 0xA5).all() and (whole[k][room + size:] == 0xA5).all(), (k, starts)
