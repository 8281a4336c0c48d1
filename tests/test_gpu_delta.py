"""GPU tests of the gated delta rule against the fp64 token loop, at every place where the
tokens and the widths are cut (chunks of 64 and 32, tiles of 16 and 32, sequence borders).

Tolerances, max |gpu - fp64| / max |fp64| of an output.  Steps on unit keys with eta <= 1 and a <= 1 do
not stretch an error.  bf16: at most five roundings of half a step (2^-8) lie on the way to an output (the
gradient of the gate: the state, its gradient, U, X and the output itself): 2e-2.  fp32: at most eight
products, of up to 128 terms of 2^-24 each: 6.2e-5.  States of bf16 problems: four operands of two terms
(2^-17 lost) and three sums of 128 terms a chunk, 5.4e-5, passed on with less than 0.7 of it a
chunk (a mean decay of 0.99 a token): 1.8e-4; without decay, 5.4e-5 for each chunk walked."""
import numpy as np
import pytest

from chunkwise_weight_recurrence_amd import binding as B
from oracle import delta_oracle as dr
from tests.block_utils import f64, rounded, torch_dtype
from tests.parity_utils import rel_err

pytestmark = pytest.mark.gpu

TOL, STATE_TOL, CHUNK_TOL = {"bf16": 2e-2, "f32": 6.2e-5}, 1.8e-4, 5.4e-5


def _unit(rng, shape, dtype):
    import torch
    x = rng.standard_normal(shape)
    return torch.from_numpy((x / np.linalg.norm(x, axis=-1, keepdims=True)).astype(np.float32)).to(torch_dtype(dtype))


def _make(seed, n, S, H, Hk, dk, dv, dtype, kind, z_mean=3.0):
    rng = np.random.default_rng(seed)
    gate = rounded(rng, (n, H), dtype, mean=z_mean, std=1.5)
    if kind == "log":
        gate = -(gate.float().abs() * 0.05).to(gate.dtype)
    return dict(q=rounded(rng, (n, Hk, dk), dtype), k=_unit(rng, (n, Hk, dk), dtype), v=rounded(rng, (n, H, dv), dtype), gate=gate,
                beta=rounded(rng, (n, H), dtype), s0=rounded(rng, (S, H, dk, dv), "f32"), d_o=rounded(rng, (n, H, dv), dtype),
                d_sf=rounded(rng, (S, H, dk, dv), "f32"))


def _train(inp, kind, dtype, starts=None, B_=None, T=None, states=True, gate=True, **kw):
    """Forward and backward on the GPU; packed with ``starts``, else dense [B_, T]."""
    import torch
    n, Hk, dk = inp["q"].shape
    H, dv = inp["v"].shape[1:]
    x = {k: v.cuda() for k, v in inp.items()}
    packed = starts is not None
    desc = B.make_delta_desc(len(starts) - 1 if packed else B_, n if packed else T, H, dk, dv, Hk=Hk, dtype=dtype,
                             gate=kind or "sigmoid", packed=packed, **kw)
    st = torch.tensor(starts, dtype=torch.int32).cuda() if packed else None
    S = desc.B

    def fresh(shape, dt):
        return torch.full(shape, float("nan"), dtype=dt, device="cuda")

    io, f32 = torch_dtype(dtype), torch.float32
    out = dict(o=fresh((n, H, dv), io), s_final=fresh((S, H, dk, dv), f32), dq=fresh((n, Hk, dk), io), dk=fresh((n, Hk, dk), io),
               dv=fresh((n, H, dv), io), dgate=fresh((n, H), io), dbeta=fresh((n, H), io), ds0=fresh((S, H, dk, dv), f32))
    size = max(B.ttt_delta_workspace_size(desc, e) for e in (0, 1))
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda") if size else None
    saved = torch.full((B.ttt_delta_saved_size(desc),), 255, dtype=torch.uint8, device="cuda")
    g, dg = (x["gate"], out["dgate"]) if gate else (None, None)
    B.ttt_delta_fwd(desc, x["q"], x["k"], x["v"], g, x["beta"], x["s0"] if states else None, st, out["o"],
                    out["s_final"] if states else None, saved, ws)
    B.ttt_delta_bwd(desc, x["q"], x["k"], x["v"], g, x["beta"], st, saved, x["d_o"], x["d_sf"] if states else None, out["dq"],
                    out["dk"], out["dv"], dg, out["dbeta"], out["ds0"] if states else None, ws)
    torch.cuda.synchronize()
    return out


def _oracle(inp, starts, kind, scale, states=True, gate=True, **kw):
    x = {k: f64(v) for k, v in inp.items()}
    g, s0, dsf = x["gate"] if gate else None, x["s0"] if states else None, x["d_sf"] if states else None
    args = (x["q"], x["k"], x["v"], g, x["beta"], starts, kind, scale)
    o, sf = dr.forward(*args, s0, **kw)
    return dict(o=o, s_final=sf, **dr.backward(*args, x["d_o"], s0, dsf, **kw))


def _check(out, want, dtype, states=True, gate=True, tol=None, state_tol=None, what=""):
    errs, bad = {}, {}
    for name, ref in want.items():
        if name in ("s_final", "ds0") and not states or name == "dgate" and not gate:
            continue
        state = name in ("s_final", "ds0")
        errs[name] = rel_err(f64(out[name]), ref)
        limit = (state_tol or (STATE_TOL if dtype == "bf16" else TOL["f32"])) if state else tol or TOL[dtype]
        if not errs[name] <= limit:
            bad[name] = errs[name]
    print(f"[delta] {what} " + " ".join(f"{k}={v:.1e}" for k, v in errs.items()), flush=True)
    assert not bad, bad


# B, T, H, Hk, dk, dv
DENSE = [(1, 1, 1, 1, 1, 1), (2, 3, 2, 1, 8, 5), (1, 16, 1, 1, 64, 64), (3, 17, 4, 2, 33, 16), (2, 31, 3, 3, 64, 48), (1, 32, 2, 2, 128, 128),
         (2, 33, 2, 1, 70, 96), (1, 63, 4, 4, 100, 7), (1, 64, 6, 2, 64, 64), (2, 65, 2, 2, 128, 64), (1, 127, 1, 1, 16, 128),
         (2, 130, 3, 1, 96, 40), (1, 300, 2, 2, 128, 128), (40, 5, 2, 2, 24, 24)]
WIDE = [(1, 70, 2, 1, 256, 256), (2, 40, 1, 1, 129, 130), (1, 66, 2, 2, 200, 64), (1, 65, 2, 2, 64, 250), (1, 64, 4, 2, 256, 33)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["sigmoid", "log"])
def test_dense(dtype, kind):
    for j, (Bn, T, H, Hk, dk, dv) in enumerate(DENSE):
        inp = _make(j, Bn * T, Bn, H, Hk, dk, dv, dtype, kind)
        states, starts = j % 3 != 2, list(range(0, Bn * T + 1, T))
        out = _train(inp, kind, dtype, B_=Bn, T=T, states=states)
        _check(out, _oracle(inp, starts, kind, dk ** -0.5, states), dtype, states, what=f"{dtype} {kind} {DENSE[j]}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_wide_heads(dtype):
    for j, (Bn, T, H, Hk, dk, dv) in enumerate(WIDE):
        inp = _make(j, Bn * T, Bn, H, Hk, dk, dv, dtype, "sigmoid")
        out = _train(inp, "sigmoid", dtype, B_=Bn, T=T)
        want = _oracle(inp, list(range(0, Bn * T + 1, T)), "sigmoid", dk ** -0.5)
        _check(out, want, dtype, tol=2 * TOL["f32"] if dtype == "f32" else None,   # products of 256 terms
               state_tol=2 * TOL["f32"] if dtype == "f32" else 2 * STATE_TOL, what=f"{dtype} {WIDE[j]}")


LENGTHS = [[1], [64], [65], [0, 0, 5, 0], [63, 1, 64, 65, 0, 130], [16] * 9, [1] * 40, [32, 33, 31, 0, 0, 1, 1, 97], [0] * 1500 + [7, 70]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_packed(dtype):
    for j, lengths in enumerate(LENGTHS):
        starts = np.concatenate([[0], np.cumsum(lengths)]).tolist()
        H, Hk, dk, dv = [(2, 1, 32, 24), (2, 2, 64, 64), (1, 1, 128, 32)][j % 3]
        if len(lengths) > 1000:
            H, Hk, dk, dv = 1, 1, 8, 8
        kind = ["sigmoid", "log"][j % 2]
        inp = _make(j, starts[-1], len(lengths), H, Hk, dk, dv, dtype, kind)
        out = _train(inp, kind, dtype, starts=starts)
        _check(out, _oracle(inp, starts, kind, dk ** -0.5), dtype, what=f"{dtype} packed {j}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_decay_and_with_larger_steps(dtype):
    n = 200
    inp = _make(5, n, 1, 2, 2, 64, 32, dtype, "sigmoid")
    inp["s0"] *= 0.3
    kw = dict(lr_max=1.5, lr_bias=-1.0, scale=0.5)
    out = _train(inp, None, dtype, B_=1, T=n, gate=False, **kw)
    okw = {k: v for k, v in kw.items() if k != "scale"}
    chunks = -(-n // (64 if dtype == "bf16" else 32))
    _check(out, _oracle(inp, [0, n], None, 0.5, gate=False, **okw), dtype, gate=False,
           state_tol=chunks * CHUNK_TOL if dtype == "bf16" else 4 * TOL["f32"], tol=4 * TOL["f32"] if dtype == "f32" else None, what=f"{dtype} no decay")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,Bn", [(1500, 1), (700, 3)])
def test_many_chunks(dtype, T, Bn):
    inp = _make(T, Bn * T, Bn, 2, 1, 64, 64, dtype, "sigmoid")
    out = _train(inp, "sigmoid", dtype, B_=Bn, T=T)
    _check(out, _oracle(inp, list(range(0, Bn * T + 1, T)), "sigmoid", 0.125), dtype, what=f"{dtype} {Bn} x {T}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,dk,dv,chunks,tail", [(1, 64, 64, 40, 1), (1, 128, 40, 67, 0), (2, 33, 96, 50, 17), (1, 256, 32, 36, 5)])
def test_long_sequences_walked_in_pieces(dtype, H, dk, dv, chunks, tail):
    """Few heads and many chunks: the forward walks pieces at the same time and joins their maps.  A map's own error,
    two-term operands as everywhere, comes to that of the states once more for each piece that is joined, passed on
    with what is left of the decay: twice the states' tolerance."""
    C = 64 if dtype == "bf16" else 32
    T, Bn = chunks * C + tail, 2 if dv == 96 else 1
    inp = _make(chunks, Bn * T, Bn, H, 1, dk, dv, dtype, "sigmoid", z_mean=5.0)
    out = _train(inp, "sigmoid", dtype, B_=Bn, T=T)
    _check(out, _oracle(inp, list(range(0, Bn * T + 1, T)), "sigmoid", dk ** -0.5), dtype,
           state_tol=4 * STATE_TOL if dtype == "bf16" else 4 * TOL["f32"], tol=4 * TOL["f32"] if dtype == "f32" else None, what=f"{dtype} pieces")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gates_at_their_ends(dtype):
    """Tokens that forget everything (a = 0) or nothing (a = 1), and steps of 0 and 1."""
    import torch
    n = 150
    for kind in ("sigmoid", "log"):
        inp = _make(11, n, 1, 2, 2, 32, 32, dtype, kind)
        end = float("-inf") if kind == "log" else -300.0
        inp["gate"][[3, 40, 63, 64, 65, 120]] = end
        inp["gate"][[5, 66]] = 0.0 if kind == "log" else 300.0
        inp["beta"][[4, 63, 100]] = -300.0
        inp["beta"][[7, 64]] = 300.0
        out = _train(inp, kind, dtype, B_=1, T=n)
        fine = {k: v.clone() for k, v in inp.items()}
        fine["gate"] = torch.where(inp["gate"] < -200, torch.full_like(inp["gate"], -200.0), inp["gate"])
        _check(out, _oracle(fine, [0, n], kind, 32 ** -0.5), dtype, what=f"{dtype} {kind} ends")
        assert (f64(out["dgate"])[[3, 64]] == 0).all() and (f64(out["dbeta"])[[4, 63, 100]] == 0).all()
    # decays so fast that a chunk's products leave fp32's range
    inp = _make(12, n, 1, 1, 1, 32, 32, dtype, "sigmoid", z_mean=-6.0)
    _check(_train(inp, "sigmoid", dtype, B_=1, T=n), _oracle(inp, [0, n], "sigmoid", 32 ** -0.5), dtype, what=f"{dtype} fast")


def test_slices_of_a_projection_at_any_offset():
    """Strided q, k, v, gate and beta, on 16 bytes or not; what lies between the slices stays."""
    import torch
    from chunkwise_weight_recurrence_amd.layer import DeltaBuffers
    rng = np.random.default_rng(3)
    for dtype, Bn, T, H, Hk, dk, dv, shift, packed in (("bf16", 2, 70, 4, 2, 64, 32, 0, False), ("bf16", 2, 70, 2, 2, 20, 30, 1, True),
                                                       ("f32", 1, 70, 2, 1, 64, 64, 3, False), ("f32", 1, 40, 2, 2, 16, 16, 0, True),
                                                       ("bf16", 1, 65, 1, 1, 128, 128, 3, False)):
        n = Bn * T
        inp = _make(9, n, Bn, H, Hk, dk, dv, dtype, "sigmoid")
        width = 2 * Hk * dk + H * dv + 2 * H
        lead = (n,) if packed else (Bn, T)
        whole = torch.full((n, width + shift + 5), 7.0, dtype=torch_dtype(dtype), device="cuda")
        parts, at = {}, shift
        for name, w, shape in (("q", Hk * dk, (Hk, dk)), ("k", Hk * dk, (Hk, dk)), ("v", H * dv, (H, dv)), ("gate", H, (H,)), ("beta", H, (H,))):
            whole[:, at:at + w] = inp[name].reshape(n, w).cuda()
            parts[name] = whole[:, at:at + w].unflatten(0, lead).unflatten(-1, shape)
            at += w
        starts = [0, T, n] if Bn == 2 else [0, n]
        st = torch.tensor(starts, dtype=torch.int32).cuda() if packed else None
        buf = DeltaBuffers(*parts.values(), s0=inp["s0"].cuda(), seq_starts=st, with_bwd=True)
        grads = torch.full_like(whole, 7.0)
        at = shift
        for name, w in (("q", Hk * dk), ("k", Hk * dk), ("v", H * dv), ("gate", H), ("beta", H)):
            setattr(buf, "d" + name, grads[:, at:at + w].unflatten(0, lead).unflatten(-1, parts[name].shape[len(lead):]))
            at += w
        buf.forward()
        buf.backward(inp["d_o"].cuda().view(*lead, H, dv), inp["d_sf"].cuda())
        torch.cuda.synchronize()
        out = {m: getattr(buf, m).reshape(n, *getattr(buf, m).shape[len(lead):]) if m not in ("s_final", "ds0") else getattr(buf, m)
               for m in ("o", "s_final", "dq", "dk", "dv", "dgate", "dbeta", "ds0")}
        _check(out, _oracle(inp, starts, "sigmoid", dk ** -0.5), dtype, what=f"{dtype} slices {shift}")
        for t in (whole, grads):
            assert (t[:, :shift] == 7).all() and (t[:, shift + width:] == 7).all()


def test_rows_of_no_sequence_and_starts_out_of_order():
    import torch
    n, H, dk, dv = 200, 2, 32, 32
    inp = _make(21, n, 3, H, H, dk, dv, "bf16", "sigmoid")
    out = _train(inp, "sigmoid", "bf16", starts=[10, 75, 75, 150])
    want = _oracle({k: (v[10:150] if v.shape[0] == n else v) for k, v in inp.items()}, [0, 65, 65, 140], "sigmoid", dk ** -0.5)
    for name in ("o", "dq", "dk", "dv", "dgate", "dbeta"):
        got = f64(out[name])
        assert np.isnan(got[:10]).all() and np.isnan(got[150:]).all(), name
        out[name] = out[name][10:150]
    _check(out, want, "bf16", what="rows of none")
    # any entries at all: nothing outside the buffers is touched, and a start below one before it counts as that one
    for starts in ([0, 5000, -3, 200], [-7, 100, 50, 1 << 30], [150, 20, 10, 0], [-5] * 4):
        out = _train(inp, "sigmoid", "bf16", starts=starts)
        edge = np.maximum.accumulate(np.clip(starts, 0, n))
        inside = np.zeros(n, bool)
        inside[edge[0]:edge[-1]] = True
        assert np.array_equal(np.isfinite(f64(out["o"])).all((1, 2)), inside)
        assert torch.isfinite(out["s_final"]).all() and torch.isfinite(out["ds0"]).all()


def test_a_nan_stays_in_its_sequence_and_head():
    n, H = 180, 2
    inp = _make(31, n, 3, H, H, 64, 32, "bf16", "sigmoid")
    starts = [0, 70, 70, 180]
    clean = _train(inp, "sigmoid", "bf16", starts=starts)
    for name, at in (("q", (20, 0, 3)), ("k", (69, 0, 1)), ("v", (0, 0, 2)), ("gate", (5, 0)), ("beta", (64, 0)), ("d_o", (69, 0, 1))):
        for bad in (float("nan"), float("inf")):
            dirty = {k: v.clone() for k, v in inp.items()}
            dirty[name][at] = bad
            out = _train(dirty, "sigmoid", "bf16", starts=starts)
            for m in ("o", "dq", "dk", "dv", "dgate", "dbeta"):
                a, b = f64(out[m]), f64(clean[m])
                assert np.array_equal(a[70:], b[70:]) and np.array_equal(a[:70, 1], b[:70, 1]), (name, m)
            for m in ("s_final", "ds0"):
                assert np.array_equal(f64(out[m])[1:], f64(clean[m])[1:]), (name, m)
            if bad != bad and name != "d_o":
                assert np.isnan(f64(out["o"])[:70, 0]).any(), name
            if name in ("gate", "beta", "k") and bad != bad:
                assert np.isnan(f64(out["s_final"])[0, 0]).any()


def test_the_same_call_gives_the_same_bits():
    inp = _make(41, 500, 1, 4, 2, 128, 128, "bf16", "sigmoid")
    a, b = (_train(inp, "sigmoid", "bf16", B_=1, T=500) for _ in range(2))
    for name in a:
        assert np.array_equal(f64(a[name]), f64(b[name])), name


def test_gradients_against_differences_on_the_gpu():
    """Central differences of <d_o, o> + <d_sf, s_final> in fp32 along random directions, h = 2^-6: what is left
    of the third order is about h^2 / 6 of the third derivative (unit directions, derivatives of order one), and the
    two losses carry 2^-24 of a sum of magnitudes near 100, over 2 h: 100 * 2^-24 / 2^-5 = 2e-4 of it."""
    import torch
    n, H, dk, dv = 90, 2, 24, 16
    inp = _make(51, n, 1, H, 1, dk, dv, "f32", "sigmoid")
    g = _train(inp, "sigmoid", "f32", B_=1, T=n)

    def loss(x):
        out = _train(x, "sigmoid", "f32", B_=1, T=n)
        return (f64(out["o"]) * f64(inp["d_o"])).sum() + (f64(out["s_final"]) * f64(inp["d_sf"])).sum()

    rng = np.random.default_rng(1)
    for name in ("q", "k", "v", "gate", "beta", "s0"):
        way = rng.standard_normal(inp[name].shape)
        way = torch.from_numpy((way / np.linalg.norm(way)).astype(np.float32))
        h = 2.0 ** -6
        got = (loss({**inp, name: inp[name] + h * way}) - loss({**inp, name: inp[name] - h * way})) / (2 * h)
        grad = f64(g["d" + name])
        want = (grad * f64(way)).sum()
        assert abs(got - want) <= 2e-3 * np.linalg.norm(grad), (name, got, want)


def test_offsets_past_32_bits():
    """Rows of 2^15 elements: the last token's lies behind 2^31 elements.  The same values close together give the same bits."""
    import torch
    from chunkwise_weight_recurrence_amd.layer import DeltaBuffers
    n, dk = 66000, 64
    inp = _make(3, n, 1, 1, 1, dk, dk, "bf16", "sigmoid")
    x = {k: inp[k].cuda()[None] for k in ("q", "k", "v", "gate", "beta", "d_o")}
    wide = torch.empty(1, n, 1 << 15, dtype=torch.bfloat16, device="cuda")
    for j, m in enumerate("qkv"):
        wide[..., dk * j:dk * (j + 1)] = x[m][..., 0, :]
    far = [wide[..., dk * j:dk * (j + 1)].unflatten(-1, (1, dk)) for j in range(3)]
    near = DeltaBuffers(x["q"], x["k"], x["v"], x["gate"], x["beta"], with_bwd=True)
    b = DeltaBuffers(*far, x["gate"], x["beta"], with_bwd=True)
    for buf in (near, b):
        buf.forward()
        buf.backward(x["d_o"])
    torch.cuda.synchronize()
    for m in ("o", "s_final", "dq", "dk", "dv", "dgate", "dbeta", "ds0"):
        assert torch.isfinite(getattr(near, m)).all() and torch.equal(getattr(near, m), getattr(b, m)), m


# ---- one token ----


def test_step_in_a_pool_past_32_bits():
    """8200 states of 16 heads of 128 x 128: the last one's lies behind 2^31 elements."""
    import torch
    H, d, states = 16, 128, 8200
    x, inp = _step_inputs(5, 2, 2, H, H, d, d, "bf16")
    pool = torch.empty(states, H, d, d, device="cuda")
    pool[-1], pool[0] = x["s0"][0], x["s0"][1]
    slots = torch.tensor([states - 1, 0], dtype=torch.int32, device="cuda")
    desc = B.make_delta_desc(2, 1, H, d, d)
    o, want = torch.empty(2, H, d, dtype=torch.bfloat16, device="cuda"), torch.empty(2, H, d, dtype=torch.bfloat16, device="cuda")
    B.ttt_delta_step(desc, x["q"], x["k"], x["v"], x["gate"], x["beta"], slots, pool, pool, o)
    small = x["s0"].clone()
    B.ttt_delta_step(desc, x["q"], x["k"], x["v"], x["gate"], x["beta"], None, small, small, want)
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(pool[-1], small[0]) and torch.equal(pool[0], small[1])


def _step_inputs(seed, rows, states, H, Hk, dk, dv, dtype):
    inp = _make(seed, rows, states, H, Hk, dk, dv, dtype, "sigmoid")
    return {k: v.cuda() for k, v in inp.items()}, inp


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,states,H,Hk,dk,dv", [(1, 1, 1, 1, 1, 1), (3, 5, 4, 2, 64, 32), (8, 8, 2, 2, 128, 128), (5, 9, 3, 1, 37, 50),
                                                    (2, 3, 2, 1, 256, 256), (300, 310, 1, 1, 16, 8), (4, 4, 2, 2, 200, 129)])
def test_step(dtype, rows, states, H, Hk, dk, dv):
    import torch
    x, inp = _step_inputs(rows, rows, states, H, Hk, dk, dv, dtype)
    x["s0"] = x["s0"][:states]
    slots = torch.randperm(states, generator=torch.Generator().manual_seed(1))[:rows].to(torch.int32)
    desc = B.make_delta_desc(rows, 1, H, dk, dv, Hk=Hk, dtype=dtype)
    o = torch.full((rows, H, dv), float("nan"), dtype=torch_dtype(dtype), device="cuda")
    new = torch.full_like(x["s0"], 9.0)
    B.ttt_delta_step(desc, x["q"], x["k"], x["v"], x["gate"], x["beta"], slots.cuda(), x["s0"], new, o)
    s = x["s0"].clone()
    o2 = torch.empty_like(o)
    B.ttt_delta_step(desc, x["q"], x["k"], x["v"], x["gate"], x["beta"], slots.cuda(), s, s, o2)
    torch.cuda.synchronize()
    at = slots.long().numpy()
    a = {k: f64(v) for k, v in inp.items()}
    want, S = dr.forward(a["q"], a["k"], a["v"], a["gate"], a["beta"], list(range(rows + 1)), "sigmoid", dk ** -0.5, a["s0"][at])
    # fp32 throughout: two sums of dk terms, the gates' few roundings, and half a step of o's type
    tol = (2 * dk + 40) * 2.0 ** -24
    assert rel_err(f64(new)[at], S) <= tol and rel_err(f64(o), want) <= tol + (2.0 ** -8 if dtype == "bf16" else 0)
    others = np.setdiff1d(np.arange(states), at)
    assert (f64(new)[others] == 9).all() and np.array_equal(f64(s)[others], f64(x["s0"])[others])
    assert np.array_equal(f64(s)[at], f64(new)[at]) and np.array_equal(f64(o), f64(o2))


def test_step_padding_and_repeated_slots():
    """Rows with one slot are its consecutive tokens; rows with none leave everything as it was."""
    import torch
    rows, H, dk, dv = 700, 2, 16, 8
    x, inp = _step_inputs(7, rows, 40, H, H, dk, dv, "f32")
    g = torch.Generator().manual_seed(3)
    slots = torch.randint(-2, 43, (rows,), generator=g).to(torch.int32)   # -2, -1, 40, 41, 42 are none
    desc = B.make_delta_desc(rows, 1, H, dk, dv, dtype="f32")
    o = torch.full((rows, H, dv), 5.0, device="cuda")
    s = x["s0"].clone()
    B.ttt_delta_step(desc, x["q"], x["k"], x["v"], x["gate"], x["beta"], slots.cuda(), s, s, o)
    torch.cuda.synchronize()
    a = {k: f64(v) for k, v in inp.items()}
    for slot in range(40):
        at = np.nonzero(slots.numpy() == slot)[0]
        want, S = dr.forward(*(a[m][at] for m in ("q", "k", "v", "gate", "beta")), [0, len(at)], "sigmoid", dk ** -0.5, a["s0"][slot:slot + 1])
        tol = (2 * dk + 40) * 2.0 ** -24 * 8   # the steps before it, each with a mean decay below 0.9
        assert rel_err(f64(s)[slot], S[0]) <= tol and (len(at) == 0 or rel_err(f64(o)[at], want) <= tol)
    none = (slots < 0) | (slots >= 40)
    assert none.any() and (o.cpu()[none] == 5).all()


def test_steps_continue_a_prefill():
    """A forward over the prompt and a step a token give what a forward over all of it gives."""
    import torch
    from chunkwise_weight_recurrence_amd.layer import DeltaBuffers
    Bn, T, more, H, dk, dv = 2, 100, 30, 2, 64, 32
    inp = _make(61, Bn * (T + more), Bn, H, 1, dk, dv, "f32", "sigmoid")
    x = {k: v.cuda().view(Bn, T + more, *v.shape[1:]) if v.shape[0] == Bn * (T + more) else v.cuda() for k, v in inp.items()}
    names = ("q", "k", "v", "gate", "beta")
    whole = DeltaBuffers(*(x[m] for m in names), s0=x["s0"])
    whole.forward()
    first = DeltaBuffers(*(x[m][:, :T].contiguous() for m in names), s0=x["s0"])
    first.forward()
    desc = B.make_delta_desc(Bn, 1, H, dk, dv, Hk=1, dtype="f32")
    s = first.s_final.clone()
    for t in range(T, T + more):
        o = torch.empty(Bn, H, dv, device="cuda")
        B.ttt_delta_step(desc, *(x[m][:, t].contiguous() for m in names), None, s, s, o)
        assert rel_err(f64(o), f64(whole.o[:, t])) <= TOL["f32"]
    assert rel_err(f64(s), f64(whole.s_final)) <= TOL["f32"]


# ---- streams and graphs ----


def _loop(seed, Bn=2, T=130, H=2, dk=64, dv=64):
    from chunkwise_weight_recurrence_amd.layer import DeltaBuffers
    inp = _make(seed, Bn * T, Bn, H, H, dk, dv, "bf16", "sigmoid")
    x = {k: v.cuda().view(Bn, T, *v.shape[1:]) if v.shape[0] == Bn * T else v.cuda() for k, v in inp.items()}
    return DeltaBuffers(x["q"], x["k"], x["v"], x["gate"], x["beta"], s0=x["s0"], with_bwd=True), x


NAMES = ("o", "s_final", "dq", "dk", "dv", "dgate", "dbeta", "ds0")


def test_a_captured_training_step_replays():
    import torch
    buf, x = _loop(71)
    other, y = _loop(72)

    def once():
        buf.forward()
        buf.backward(x["d_o"], x["d_sf"])

    def eager(src):   # on buffers of its own
        b = type(buf)(src["q"], src["k"], src["v"], src["gate"], src["beta"], s0=src["s0"], with_bwd=True)
        b.forward()
        b.backward(src["d_o"], src["d_sf"])
        return {m: getattr(b, m).clone() for m in NAMES}

    wants = [eager(x), eager(y)]
    first = {k: v.clone() for k, v in x.items()}
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        once()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        once()
    for k in range(4):
        for m in x:
            x[m].copy_((first, y)[k % 2][m])
        for m in NAMES:
            getattr(buf, m).fill_(float("nan"))
        buf.ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(getattr(buf, m), wants[k % 2][m]) for m in NAMES), k
        eager(y)


def test_two_streams_with_a_workspace_each():
    import torch
    work = []
    for seed in (81, 82, 83):
        b, x = _loop(seed, T=400)
        b.forward()
        b.backward(x["d_o"], x["d_sf"])
        work.append((b, x, {m: getattr(b, m).clone() for m in NAMES}, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for b, x, _, s in work:
        for m in NAMES:
            getattr(b, m).fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(3):
        for b, x, _, s in work:
            b.forward(stream=s)
            b.backward(x["d_o"], x["d_sf"], stream=s)
    torch.cuda.synchronize()
    for b, _, want, _ in work:
        assert all(torch.equal(getattr(b, m), want[m]) for m in NAMES)


def test_a_captured_decode_step_takes_new_rows():
    import torch
    rows, H, dk, dv = 5, 2, 64, 64
    x, _ = _step_inputs(91, rows, 8, H, H, dk, dv, "bf16")
    slots = torch.tensor([3, 0, 7, -1, 5], dtype=torch.int32, device="cuda")
    desc = B.make_delta_desc(rows, 1, H, dk, dv)
    o, s = torch.zeros(rows, H, dv, dtype=torch.bfloat16, device="cuda"), x["s0"].clone()
    step = lambda s_, o_: B.ttt_delta_step(desc, x["q"], x["k"], x["v"], x["gate"], x["beta"], slots, s_, s_, o_)  # noqa: E731
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(s.clone(), o.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(s, o)
    want, o_want = x["s0"].clone(), torch.zeros_like(o)
    g = torch.Generator(device="cuda").manual_seed(1)
    for _ in range(5):
        x["v"].normal_(generator=g)
        slots.copy_(torch.randperm(9, generator=g, device="cuda")[:rows].to(torch.int32))   # 8 is none
        step(want, o_want)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(s, want) and torch.equal(o, o_want)


# ---- together ----


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("packed", [False, True])
def test_block_of_norm_rotation_rule_and_norm(dtype, packed):
    """Queries and keys normed and rotated, the rule over them, a layer norm per head, forward and backward.  fp32: the
    norms add a gain below 3 each: 9 times the rule's tolerance.  bf16: as the rule's, with the roundings of the normed q, k
    and their gradients on the way: seven of 2^-8."""
    import torch
    from chunkwise_weight_recurrence_amd.layer import DeltaBuffers, LayerNormBuffers, QkNormBuffers
    from oracle import layernorm_oracle as ln
    from oracle import qknorm_oracle as qk
    Bn, T, H, Hk, dk, dv = 2, 140, 4, 2, 32, 24
    n = Bn * T
    lead = (n,) if packed else (Bn, T)
    starts = [0, 100, 100, 260, n] if packed else [0, T, n]
    rng = np.random.default_rng(0)
    inp = _make(0, n, 1, H, Hk, dk, dv, dtype, "sigmoid")
    q, k = rounded(rng, (n, Hk, dk), dtype, std=2.0), rounded(rng, (n, Hk, dk), dtype, std=3.0)
    pos = rng.integers(0, 5000, n).astype(np.int32)
    freq = (100.0 ** -np.arange(8)).astype(np.float32)
    w, b = rounded(rng, (H, dv), "f32", mean=1.0, std=0.2), rounded(rng, (H, dv), "f32", std=0.2)
    dy = rounded(rng, (n * H, dv), dtype)
    at = lambda t: t.cuda().view(*lead, *t.shape[1:])  # noqa: E731
    st = torch.tensor(starts, dtype=torch.int32).cuda() if packed else None
    pre = QkNormBuffers(at(q), at(k), positions=torch.from_numpy(pos).cuda(), inv_freq=torch.from_numpy(freq).cuda(), norm="l2", with_bwd=True)
    mix = DeltaBuffers(pre.yq, pre.yk, at(inp["v"]), at(inp["gate"]), at(inp["beta"]), seq_starts=st, with_bwd=True)
    post = LayerNormBuffers(mix.o.view(n * H, dv), w.cuda(), b.cuda(), groups=H, period=1, with_bwd=True)
    pre.forward()
    mix.forward()
    post.forward()
    post.backward(dy.cuda())
    mix.backward(post.dx.view(*lead, H, dv))
    pre.backward(mix.dq, mix.dk)
    torch.cuda.synchronize()
    got = dict(y=post.y, dq=pre.dq, dk=pre.dk, dv=mix.dv, dgate=mix.dgate, dbeta=mix.dbeta, dw=post.dw, db=post.db)
    yq, yk = (qk.forward(f64(x), None, pos, freq, "l2", "half") for x in (q, k))
    args = (yq, yk, f64(inp["v"]), f64(inp["gate"]), f64(inp["beta"]), starts, "sigmoid", dk ** -0.5)
    o, _ = dr.forward(*args)
    f = ln.forward(o.reshape(n * H, dv), f64(w), f64(b), 1e-5, H, 1)
    g = ln.backward(o.reshape(n * H, dv), f64(w), 1e-5, f64(dy), None, H, 1)
    gm = dr.backward(*args, g["dx"].reshape(n, H, dv))
    want = dict(y=f["y"], dv=gm["dv"], dgate=gm["dgate"], dbeta=gm["dbeta"], dw=g["dw"], db=g["db"])
    for name, x in (("dq", q), ("dk", k)):
        want[name] = qk.backward(f64(x), None, pos, freq, "l2", "half", gm[name])[0]
    errs = {m: rel_err(f64(got[m]).reshape(want[m].shape), want[m]) for m in want}
    print(f"[block] {dtype} packed={packed} " + " ".join(f"{m}={e:.1e}" for m, e in errs.items()), flush=True)
    assert all(e <= (7 * 2.0 ** -8 if dtype == "bf16" else 9 * TOL["f32"]) for e in errs.values()), errs
