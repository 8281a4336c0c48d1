"""GPU tests of the norm and rotation of queries and keys against the fp64 oracle.

Tolerances, for each value against its row's size: an output is a turned pair of normed values, so
fp32 arithmetic is off by at most (d + 20) 2^-24 of the row's largest value (the sum of squares d terms, half of
which the root passes on; the angle, reduced in 64 bits, 2^-24 of a turn's 2 pi; the two products) and the
output's rounding by half a step.  dx adds one more sum over the row."""
import numpy as np
import pytest

from chunkwise_weight_recurrence_amd import binding as B
from oracle import qknorm_oracle as qk
from tests.block_utils import HALF, f64, rounded, torch_dtype

pytestmark = pytest.mark.gpu


def _row_err(got, ref):
    """max |got - ref| over the largest value of the row."""
    got, ref = f64(got).reshape(ref.shape), np.asarray(ref)
    if got.size == 0:
        return 0.0
    assert np.isfinite(got).all()
    size = np.abs(ref).max(-1, keepdims=True)
    return float((np.abs(got - ref) / np.where(size > 0, size, 1.0)).max())


def _make(seed, n, Hq, Hk, d, rot, dtype, weight, far):
    import torch
    rng = np.random.default_rng(seed)
    scale = np.exp(rng.normal(0, 1, (n, 1, 1)))
    inp = dict(q=rounded(rng, (n, Hq, d), "f32") * torch.from_numpy(scale.astype(np.float32)), k=rounded(rng, (n, Hk, d), "f32", std=0.3))
    inp = {m: x.to(torch_dtype(dtype)) for m, x in inp.items()}
    inp.update(dyq=rounded(rng, (n, Hq, d), dtype), dyk=rounded(rng, (n, Hk, d), dtype))
    inp["wq"] = rounded(rng, (d,), "f32", mean=1.0, std=0.3) if weight else None
    inp["wk"] = rounded(rng, (d,), "f32", mean=1.0, std=0.3) if weight else None
    inp["pos"] = torch.from_numpy(rng.integers(-10, 2_000_000_000 if far else 4000, n).astype(np.int32))
    inp["freq"] = torch.from_numpy((1e4 ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32))
    return inp


def _run(inp, dtype, norm, pairing, eps, scale, **kw):
    import torch
    n, Hq, d = inp["q"].shape
    Hk = inp["k"].shape[1]
    x = {m: v if v is None else v.cuda() for m, v in inp.items()}
    rot = 2 * inp["freq"].numel()
    desc = B.make_qknorm_desc(n, Hq, Hk, d, rot=rot, pairing=pairing, norm=norm, dtype=dtype, eps=eps, rot_scale=scale, **kw)
    io = torch_dtype(dtype)
    fresh = lambda x, t=io: torch.full(x.shape, float("nan"), dtype=t, device="cuda")  # noqa: E731
    out = dict(yq=fresh(inp["q"]), yk=fresh(inp["k"]), dq=fresh(inp["q"]), dk=fresh(inp["k"]))
    f = torch.float32
    out.update(dwq=torch.full((d,), float("nan"), dtype=f, device="cuda"), dwk=torch.full((d,), float("nan"), dtype=f, device="cuda"))
    ws = torch.full((B.ttt_qknorm_workspace_size(desc),), 255, dtype=torch.uint8, device="cuda")
    freq = x["freq"] if rot else None
    k, dyk, yk, dk = (x["k"], x["dyk"], out["yk"], out["dk"]) if Hk else (None,) * 4
    B.ttt_qknorm_fwd(desc, x["q"], k, x["wq"], x["wk"], x["pos"], freq, out["yq"], yk)
    B.ttt_qknorm_bwd(desc, x["q"], k, x["wq"], x["wk"], x["pos"], freq, x["dyq"], dyk, out["dq"], dk, out["dwq"], out["dwk"], ws)
    torch.cuda.synchronize()
    return out


def _check(inp, out, dtype, norm, pairing, eps, scale, pos=None):
    d = inp["q"].shape[-1]
    pos = inp["pos"].numpy() if pos is None else pos
    unit = (d + 20) * 2.0 ** -24
    for m in "qk":
        x = f64(inp[m])
        w = None if inp["w" + m] is None else f64(inp["w" + m])
        args = (x, w, pos, f64(inp["freq"]), norm, pairing)
        y = qk.forward(*args, eps=eps, scale=scale)
        dx, dw = qk.backward(*args, f64(inp["dy" + m]), eps=eps, scale=scale)
        assert _row_err(out["y" + m], y) <= 2 * unit + HALF[dtype], (m, _row_err(out["y" + m], y))
        # dx is a difference: against the size of what is taken apart, r |w dz|
        h, r = qk._hat(x, norm, eps)
        dz = qk.turn(f64(inp["dy" + m]), pos, f64(inp["freq"]), pairing, scale, back=True)
        size = np.abs(r * dz * (1 if w is None else w)).max(-1, keepdims=True) * 2
        err = np.abs(f64(out["d" + m]) - dx) / np.where(size > 0, size, 1) if dx.size else np.zeros(1)
        assert err.max() <= 4 * unit + HALF[dtype], (m, err.max())
        # a column's sum: each term off by a few units of the largest, added up in slots of rows and a tree
        terms = np.abs(dz * h).sum((0, 1))
        assert (np.abs(f64(out["dw" + m]) - dw) <= (64 + d) * 2.0 ** -24 * terms + 1e-30).all(), m


# tokens, Hq, Hk, d, rot
SHAPES = [(1, 1, 1, 1, 0), (1, 1, 1, 2, 2), (3, 4, 2, 64, 64), (5, 2, 1, 128, 64), (7, 3, 3, 80, 48), (2, 1, 1, 256, 256), (9, 5, 1, 70, 34),
          (33, 8, 2, 16, 16), (4, 2, 2, 512, 512), (3, 2, 1, 333, 100), (70, 20, 20, 96, 96), (6, 1, 1, 24, 8), (11, 2, 2, 40, 16), (130, 1, 0, 64, 32),
          (2, 3, 1, 511, 510), (300, 16, 4, 128, 128), (5000, 1, 1, 8, 8), (4, 2, 2, 136, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("norm", ["rms", "l2", "none"])
@pytest.mark.parametrize("pairing", ["half", "interleaved"])
def test_against_the_oracle(dtype, norm, pairing):
    for j, (n, Hq, Hk, d, rot) in enumerate(SHAPES):
        inp = _make(j, n, Hq, Hk, d, rot, dtype, j % 2 == 0, j % 3 == 0)
        eps, scale = (1e-6, 1.0) if j % 2 else (1e-3, 1.25)
        out = _run(inp, dtype, norm, pairing, eps, scale)
        print(f"[qknorm] {dtype} {norm} {pairing} {SHAPES[j]}", flush=True)
        _check(inp, out, dtype, norm, pairing, eps, scale)


def test_positions_by_period():
    import torch
    inp = _make(3, 50, 2, 2, 64, 64, "f32", True, False)
    for period, pos in ((0, np.arange(50)), (7, np.arange(50) % 7)):
        x = {**inp, "pos": None}
        n, Hq, d = inp["q"].shape
        out = _run(x, "f32", "rms", "half", 1e-6, 1.0, period=period)
        _check(inp, out, "f32", "rms", "half", 1e-6, 1.0, pos=pos)
    assert torch.isfinite(out["yq"]).all()


def test_slices_in_place_and_rows_of_zeros():
    import torch
    from chunkwise_weight_recurrence_amd.layer import QkNormBuffers
    inp = _make(4, 30, 4, 2, 64, 32, "bf16", True, False)
    for shift in (0, 8, 3):
        whole = torch.full((30, 6 * 64 + shift + 9), 7.0, dtype=torch.bfloat16, device="cuda")
        whole[:, shift:shift + 256] = inp["q"].reshape(30, 256).cuda()
        whole[:, shift + 256:shift + 384] = inp["k"].reshape(30, 128).cuda()
        q, k = whole[:, shift:shift + 256].unflatten(-1, (4, 64)), whole[:, shift + 256:shift + 384].unflatten(-1, (2, 64))
        buf = QkNormBuffers(q, k, inp["wq"].cuda(), inp["wk"].cuda(), inp["pos"].cuda(), inp["freq"].cuda(), with_bwd=True)
        grads = torch.full_like(whole, 7.0)
        buf.dq, buf.dk = grads[:, shift:shift + 256].unflatten(-1, (4, 64)), grads[:, shift + 256:shift + 384].unflatten(-1, (2, 64))
        buf.forward()
        buf.backward(inp["dyq"].cuda(), inp["dyk"].cuda())
        torch.cuda.synchronize()
        out = {m: getattr(buf, m) for m in ("yq", "yk", "dq", "dk", "dwq", "dwk")}
        _check(inp, out, "bf16", "rms", "half", 1e-6, 1.0)
        for t in (whole, grads):
            assert (t[:, :shift] == 7).all() and (t[:, shift + 384:] == 7).all()
    # in place, and a row of zeros (eps alone keeps it finite)
    q, k = inp["q"].cuda(), inp["k"].cuda()
    q[3] = 0
    desc = B.make_qknorm_desc(30, 4, 2, 64, rot=32)
    yq, yk = torch.empty_like(q), torch.empty_like(k)
    B.ttt_qknorm_fwd(desc, q, k, None, None, inp["pos"].cuda(), inp["freq"].cuda(), yq, yk)
    B.ttt_qknorm_fwd(desc, q, k, None, None, inp["pos"].cuda(), inp["freq"].cuda(), q, k)
    torch.cuda.synchronize()
    assert torch.equal(q, yq) and torch.equal(k, yk) and (yq[3] == 0).all()


def test_nan_and_infinity_stay_in_their_row():
    import torch
    inp = _make(5, 12, 4, 2, 64, 64, "bf16", False, False)
    clean = _run(inp, "bf16", "rms", "half", 1e-6, 1.0)
    for bad in (float("nan"), float("inf")):
        dirty = {**inp, "q": inp["q"].clone()}
        dirty["q"][2, 1, 5] = bad
        out = _run(dirty, "bf16", "rms", "half", 1e-6, 1.0)
        for m in ("yq", "dq"):
            a, b = out[m].clone(), clean[m].clone()
            assert torch.isnan(a[2, 1]).any()
            a[2, 1] = b[2, 1] = 0
            assert torch.equal(a, b)
        assert torch.equal(out["yk"], clean["yk"]) and torch.equal(out["dk"], clean["dk"])


def test_no_tokens_and_no_weights_wanted():
    import torch
    inp = _make(6, 0, 2, 1, 16, 16, "f32", True, False)
    out = _run(inp, "f32", "rms", "half", 1e-6, 1.0)
    assert (out["dwq"] == 0).all() and (out["dwk"] == 0).all()
    inp = _make(7, 6, 2, 1, 16, 16, "f32", True, False)
    x = {m: v.cuda() for m, v in inp.items()}
    desc = B.make_qknorm_desc(6, 2, 1, 16, dtype="f32")
    dq, dk = torch.empty_like(x["q"]), torch.empty_like(x["k"])
    B.ttt_qknorm_bwd(desc, x["q"], x["k"], x["wq"], x["wk"], x["pos"], x["freq"], x["dyq"], x["dyk"], dq, dk, None, None, None)
    want = _run(inp, "f32", "rms", "half", 1e-6, 1.0)
    torch.cuda.synchronize()
    assert torch.equal(dq, want["dq"]) and torch.equal(dk, want["dk"])


def test_captured_and_on_two_streams():
    import torch
    from chunkwise_weight_recurrence_amd.layer import QkNormBuffers

    def make(seed):
        inp = _make(seed, 200, 8, 4, 64, 64, "bf16", True, False)
        x = {m: v.cuda() for m, v in inp.items()}
        return QkNormBuffers(x["q"], x["k"], x["wq"], x["wk"], x["pos"], x["freq"], with_bwd=True), x

    names = ("yq", "yk", "dq", "dk", "dwq", "dwk")
    work = []
    for seed in (1, 2):
        b, x = make(seed)
        b.forward()
        b.backward(x["dyq"], x["dyk"])
        work.append((b, x, {m: getattr(b, m).clone() for m in names}, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for b, x, _, s in work:
        b.forward(stream=s)
        b.backward(x["dyq"], x["dyk"], stream=s)
    torch.cuda.synchronize()
    for b, _, want, _ in work:
        assert all(torch.equal(getattr(b, m), want[m]) for m in names)
    b, x, want, side = work[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        b.forward()
        b.backward(x["dyq"], x["dyk"])
    for k in range(4):
        for m in names:
            getattr(b, m).fill_(float("nan"))
        b.ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(getattr(b, m), want[m]) for m in names), k
        work[1][0].forward()


def test_offsets_past_32_bits():
    """Rows of 2^15 elements: the last token's lies behind 2^31 elements.  The same values close together give the same bits."""
    import torch
    from chunkwise_weight_recurrence_amd.layer import QkNormBuffers
    n, d = 66000, 64
    inp = _make(9, n, 1, 1, d, d, "bf16", True, False)
    x = {m: v.cuda() for m, v in inp.items()}
    wide = torch.empty(n, 1 << 15, dtype=torch.bfloat16, device="cuda")
    wide[:, :d], wide[:, d:2 * d] = x["q"][:, 0], x["k"][:, 0]
    rest = (x["wq"], x["wk"], x["pos"], x["freq"])
    near = QkNormBuffers(x["q"], x["k"], *rest, with_bwd=True)
    far = QkNormBuffers(wide[:, None, :d], wide[:, None, d:2 * d], *rest, with_bwd=True)
    for b in (near, far):
        b.forward()
        b.backward(x["dyq"], x["dyk"])
    torch.cuda.synchronize()
    for m in ("yq", "yk", "dq", "dk", "dwq", "dwk"):
        assert torch.isfinite(getattr(near, m)).all() and torch.equal(getattr(near, m), getattr(far, m)), m
