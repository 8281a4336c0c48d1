"""GPU tests of the layer norm against the fp64 oracle: every way a row is laid over
threads, grouped weights, residuals, strides, and rows that are hard to normalise.

Tolerances: the oracle's bound on fp32 arithmetic plus half a step of the output's
type (``tests/block_utils.py::worst``; above 1 is wrong)."""
import numpy as np
import pytest

from chunkwise_weight_recurrence_amd import binding as B
from oracle import layernorm_oracle as ln
from tests.block_utils import f64, rounded, torch_dtype, worst

pytestmark = pytest.mark.gpu

EPS = 1e-5


def _run(rows, D, dtype, groups=1, period=1, residual=False, affine=True, seed=0, x=None, dr=True, eps=EPS):
    import torch
    rng = np.random.default_rng(seed)
    x = rounded(rng, (rows, D), dtype, mean=0.5, std=2.0) if x is None else x
    res = rounded(rng, (rows, D), dtype) if residual else None
    w = rounded(rng, (groups, D), "f32", mean=1.0, std=0.3) if affine else None
    b = rounded(rng, (groups, D), "f32") if affine else None
    dy = rounded(rng, (rows, D), dtype)
    drt = rounded(rng, (rows, D), dtype) if dr else None
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    io = dict(dtype=torch_dtype(dtype), device="cuda")
    f32 = dict(dtype=torch.float32, device="cuda")
    nan = float("nan")
    out = dict(y=torch.full((rows, D), nan, **io), mean=torch.full((rows,), nan, **f32), rstd=torch.full((rows,), nan, **f32),
               dx=torch.full((rows, D), nan, **io), dw=torch.full((groups, D), nan, **f32), db=torch.full((groups, D), nan, **f32))
    r = torch.full((rows, D), nan, **io) if residual else None
    desc = B.make_ln_desc(rows, D, dtype=dtype, groups=groups, period=period, eps=eps)
    ws = torch.full((B.ttt_layernorm_workspace_size(desc),), 255, dtype=torch.uint8, device="cuda")
    xd = dev(x)
    B.ttt_layernorm_fwd(desc, xd, dev(res), dev(w), dev(b), out["y"], r, out["mean"], out["rstd"])
    kept = r if residual else xd
    B.ttt_layernorm_bwd(desc, kept, dev(w), out["mean"], out["rstd"], dev(dy), dev(drt), out["dx"], out["dw"], out["db"], ws)
    torch.cuda.synchronize()
    if residual:
        assert torch.equal(r.cpu(), (x.float() + res.float()).to(x.dtype))
    f = ln.forward(f64(kept), None if w is None else f64(w), None if b is None else f64(b), eps, groups, period)
    g = ln.backward(f64(kept), None if w is None else f64(w), eps, f64(dy), f64(drt) if dr else None, groups, period)
    errs = dict(y=worst(out["y"], f["y"], f["e_y"], dtype), mean=worst(out["mean"], f["mean"], f["e_mean"], "f32"),
                rstd=worst(out["rstd"], f["rstd"], f["e_rstd"], "f32"), dx=worst(out["dx"], g["dx"], g["e_dx"], dtype),
                dw=worst(out["dw"], g["dw"], g["e_dw"], "f32"), db=worst(out["db"], g["db"], g["e_db"], "f32"))
    assert all(e <= 1.0 for e in errs.values()), ((rows, D, dtype, groups, period), errs)
    return out


# narrow rows (a part of a wave), a whole wave, several waves; one piece a thread in each
WIDTHS = [1, 2, 7, 8, 16, 24, 63, 64, 65, 128, 130, 256, 500, 512, 513, 520, 1000, 1001, 1024, 2048, 2560, 4000]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_widths(dtype):
    for k, D in enumerate(WIDTHS):
        for rows in (1, 3, 37):
            _run(rows, D, dtype, residual=k % 2 == 0, affine=k % 3 != 0, seed=k, dr=k % 2 == 1)


@pytest.mark.parametrize("D,dtype", [(4104, "bf16"), (8192, "bf16"), (9000, "f32"), (20000, "bf16"), (20001, "f32"),
                                     (32768, "bf16")])
def test_wide_rows(D, dtype):
    _run(5, D, dtype, residual=D % 2 == 0)


# One row of a slot at a time: several at a time need 4096 rows a slot (test_rows_of_a_slot_together).
@pytest.mark.parametrize("rows,D,dtype", [(20000, 24, "bf16"), (9001, 128, "bf16"), (5003, 520, "f32"), (8200, 33, "f32")])
def test_many_rows(rows, D, dtype):
    """Several steps of a workgroup, four rows at a time, a ragged last one."""
    _run(rows, D, dtype, residual=True)


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 600), ("f32", 30)])
def test_grouped_weights(dtype, D):
    for groups, period, reps in ((2, 1, 5), (3, 7, 1), (16, 5, 3), (5, 300, 2), (700, 1, 2)):
        _run(groups * period * reps, D, dtype, groups=groups, period=period)


def test_wide_grouped_rows():
    _run(12, 20001, "bf16", groups=2, period=3)


def test_means_far_above_the_deviation():
    """Rows around 1000 with a deviation of 1: the variance must not be a difference of large squares."""
    import torch
    rng = np.random.default_rng(3)
    for D in (96, 1001, 20001):
        _run(40, D, "f32", x=rounded(rng, (40, D), "f32", mean=1000.0), seed=1)
        spike = rounded(rng, (40, D), "bf16")
        spike[:, 0] = 3000.0   # one channel far out
        _run(40, D, "bf16", x=spike, seed=2)
    # constant rows: only eps is left under the root
    x = torch.full((5, 64), 2.0, dtype=torch.bfloat16)
    out = _run(5, 64, "bf16", x=x, seed=3)
    assert torch.allclose(out["rstd"].cpu(), torch.full((5,), EPS ** -0.5), rtol=1e-6)


def test_bad_rows_stay_alone():
    import torch
    rng = np.random.default_rng(4)
    for D in (64, 1000, 20001):
        x = rounded(rng, (9, D), "bf16")
        desc = B.make_ln_desc(9, D)
        ys = []
        for bad in (None, float("nan"), float("inf")):
            v = x.clone()
            if bad is not None:
                v[4, D // 2] = bad
            y = torch.empty_like(v, device="cuda")
            B.ttt_layernorm_fwd(desc, v.cuda(), None, None, None, y, None, None, None)
            ys.append(y.cpu())
        good = [i for i in range(9) if i != 4]
        for y in ys[1:]:
            assert torch.equal(y[good], ys[0][good]) and torch.isnan(y[4]).any()


def test_no_rows():
    import torch
    desc = B.make_ln_desc(0, 64, groups=2)
    dw, db = (torch.full((2, 64), float("nan"), device="cuda") for _ in range(2))
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    m = torch.empty(0, device="cuda")
    ws = torch.empty(B.ttt_layernorm_workspace_size(desc), dtype=torch.uint8, device="cuda")
    B.ttt_layernorm_fwd(desc, e, None, None, None, e, None, m, m)
    B.ttt_layernorm_bwd(desc, e, None, m, m, e, None, e, dw, db, ws)
    torch.cuda.synchronize()
    assert (dw == 0).all() and (db == 0).all()   # a sum over nothing


def test_optional_outputs():
    """dw alone, db alone, neither (then without a workspace); inference without mean and rstd."""
    import torch
    out = _run(50, 200, "bf16", seed=5)
    rng = np.random.default_rng(5)
    x = rounded(rng, (50, 200), "bf16", mean=0.5, std=2.0).cuda()
    w = rounded(rng, (1, 200), "f32", mean=1.0, std=0.3).cuda()
    b = rounded(rng, (1, 200), "f32").cuda()
    dy, dr = (rounded(rng, (50, 200), "bf16").cuda() for _ in range(2))
    desc = B.make_ln_desc(50, 200)
    y = torch.empty_like(x)
    B.ttt_layernorm_fwd(desc, x, None, w, b, y, None, None, None)
    assert torch.equal(y, out["y"])
    ws = torch.empty(B.ttt_layernorm_workspace_size(desc), dtype=torch.uint8, device="cuda")
    for want_w, want_b in ((True, False), (False, True), (False, False)):
        dx = torch.empty_like(x)
        dw, db = (torch.empty_like(w) if q else None for q in (want_w, want_b))
        B.ttt_layernorm_bwd(desc, x, w, out["mean"], out["rstd"], dy, dr, dx, dw, db, ws if want_w or want_b else None)
        assert torch.equal(dx, out["dx"])
        assert dw is None or torch.equal(dw, out["dw"])
        assert db is None or torch.equal(db, out["db"])


def test_strided_rows_and_residual_in_place():
    import torch
    from chunkwise_weight_recurrence_amd.layer import LayerNormBuffers
    rng = np.random.default_rng(6)
    for D, room in ((64, 200), (33, 47), (600, 1208)):
        wide = torch.full((4, 10, room), float("nan"), dtype=torch.bfloat16, device="cuda")
        x = wide[..., :D]
        x.copy_(rounded(rng, (4, 10, D), "bf16"))
        w = rounded(rng, (1, D), "f32").cuda()
        dy = rounded(rng, (4, 10, D), "bf16").cuda()
        buf = LayerNormBuffers(x, w, with_bwd=True)
        dwide = torch.full_like(wide, 7.0)
        buf.dx = dwide[..., :D]
        buf.forward()
        buf.backward(dy)
        dense = LayerNormBuffers(x.contiguous(), w, with_bwd=True)
        dense.forward()
        dense.backward(dy)
        f = ln.forward(f64(x).reshape(40, D), f64(w), None, EPS)
        g = ln.backward(f64(x).reshape(40, D), f64(w), EPS, f64(dy).reshape(40, D))
        assert worst(buf.y.reshape(40, D), f["y"], f["e_y"], "bf16") <= 1
        assert worst(buf.dx.reshape(40, D), g["dx"], g["e_dx"], "bf16") <= 1 and worst(buf.dw, g["dw"], g["e_dw"], "f32") <= 1
        assert (dwide[..., D:] == 7.0).all()
        # the residual stream updated in place
        stream = rounded(rng, (4, 10, D), "bf16").cuda()
        apart = LayerNormBuffers(x, w, res=stream.clone())
        apart.forward()
        same = LayerNormBuffers(x, w, res=stream)
        same.r = stream
        same.forward()
        assert torch.equal(same.y, apart.y) and torch.equal(stream, apart.r)


@pytest.mark.parametrize("D,dtype", [(9, "bf16"), (5, "f32"), (515, "bf16"), (1027, "bf16"), (8191, "bf16"), (8193, "bf16"),
                                     (16385, "bf16"), (24575, "bf16"), (24577, "bf16"), (4099, "f32"), (8194, "f32"),
                                     (12291, "f32"), (20479, "f32"), (20481, "f32")])
def test_rows_that_end_inside_a_piece(D, dtype):
    """The last piece of a row reaches back over its neighbour: each element counts once and
    is kept, with rows beyond the first of a workgroup and the residual stream in place."""
    import torch
    rows = 300 if D > 64 else 9001
    out = _run(rows, D, dtype, residual=True, seed=10)
    rng = np.random.default_rng(10)
    x, res = rounded(rng, (rows, D), dtype, mean=0.5, std=2.0).cuda(), rounded(rng, (rows, D), dtype).cuda()
    w, b = rounded(rng, (1, D), "f32", mean=1.0, std=0.3).cuda(), rounded(rng, (1, D), "f32").cuda()
    kept, y = (x.float() + res.float()).to(x.dtype), torch.empty_like(x)
    B.ttt_layernorm_fwd(B.make_ln_desc(rows, D, dtype=dtype, eps=EPS), x, res, w, b, y, res, None, None)
    assert torch.equal(y, out["y"]) and torch.equal(res, kept)


@pytest.mark.parametrize("D", [33, 1001, 20001])
def test_infinity_in_the_last_columns(D):
    """An infinity where two pieces overlap: the mean is infinite, not NaN, and other rows are untouched."""
    import torch
    rng = np.random.default_rng(11)
    x = rounded(rng, (5, D), "bf16")
    desc = B.make_ln_desc(5, D)
    means = []
    for bad in (None, 0, D - 1, D - 2, D - 7):
        v = x.clone()
        if bad is not None:
            v[2, bad] = float("inf")
        mean, y = torch.empty(5, device="cuda"), torch.empty_like(v, device="cuda")
        B.ttt_layernorm_fwd(desc, v.cuda(), None, None, None, y, None, mean, None)
        means.append(mean.cpu())
    for m in means[1:]:
        assert m[2] == float("inf") and torch.equal(m[[0, 1, 3, 4]], means[0][[0, 1, 3, 4]])


def test_repeats_to_the_bit():
    import torch
    a = _run(9000, 128, "bf16", groups=4, period=750, seed=7)
    for _ in range(3):
        b = _run(9000, 128, "bf16", groups=4, period=750, seed=7)
        assert all(torch.equal(a[k], b[k]) for k in a)


def test_offsets_past_32_bits():
    import torch
    rows, D = 70_000, 32_768   # 2.3e9 elements
    rng = np.random.default_rng(8)
    x = torch.zeros((rows, D), dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros_like(x)
    tail, dt = rounded(rng, (40, D), "bf16"), rounded(rng, (40, D), "bf16")
    x[-40:], dy[-40:] = tail.cuda(), dt.cuda()
    w = rounded(rng, (1, D), "f32")
    desc = B.make_ln_desc(rows, D)
    y = torch.empty_like(x)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dw, db = torch.empty(1, D, device="cuda"), torch.empty(1, D, device="cuda")
    ws = torch.empty(B.ttt_layernorm_workspace_size(desc), dtype=torch.uint8, device="cuda")
    B.ttt_layernorm_fwd(desc, x, None, w.cuda(), None, y, None, mean, rstd)
    f = ln.forward(f64(tail), f64(w), None, EPS)
    assert worst(y[-40:], f["y"], f["e_y"], "bf16") <= 1 and not y[:-40].any()
    B.ttt_layernorm_bwd(desc, x, w.cuda(), mean, rstd, dy, None, y, dw, db, ws)
    g = ln.backward(f64(tail), f64(w), EPS, f64(dt))
    assert worst(y[-40:], g["dx"], g["e_dx"], "bf16") <= 1 and not y[:-40].any()
    assert worst(dw, g["dw"], g["e_dw"], "f32") <= 1 and worst(db, g["db"], g["e_db"], "f32") <= 1


def test_a_weight_of_many_groups():
    """More columns of dw and db than one launch of the reduction has workgroups for: two rows a group."""
    import torch
    G, D = 1 << 20, 72
    gen = torch.Generator(device="cuda").manual_seed(12)
    x, dy = (torch.randn(2 * G, D, device="cuda", dtype=torch.bfloat16, generator=gen) for _ in range(2))
    w = torch.randn(G, D, device="cuda", generator=gen)
    desc = B.make_ln_desc(2 * G, D, groups=G, eps=EPS)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = (torch.empty(2 * G, device="cuda") for _ in range(2))
    dw, db = torch.empty_like(w), torch.empty_like(w)
    ws = torch.empty(B.ttt_layernorm_workspace_size(desc), dtype=torch.uint8, device="cuda")
    B.ttt_layernorm_fwd(desc, x, None, w, None, y, None, mean, rstd)
    B.ttt_layernorm_bwd(desc, x, w, mean, rstd, dy, None, dx, dw, db, ws)
    for g0 in (0, 5, 466_000, 466_033, 932_060, G - 4):   # 2^25 columns are 233 016.9 groups' dw and db
        rows = torch.cat([torch.arange(g0, g0 + 4), torch.arange(G + g0, G + g0 + 4)])
        part = rows.cuda()
        want = ln.backward(f64(x[part]), f64(w[g0:g0 + 4]), EPS, f64(dy[part]), None, 4, 1)
        assert worst(dw[g0:g0 + 4], want["dw"], want["e_dw"], "f32") <= 1
        assert worst(db[g0:g0 + 4], want["db"], want["e_db"], "f32") <= 1
        assert worst(dx[part], want["dx"], want["e_dx"], "bf16") <= 1


def test_graph_replays():
    import torch
    from chunkwise_weight_recurrence_amd.layer import LayerNormBuffers
    rng = np.random.default_rng(9)
    probs = []
    for rows, D, G in ((600, 200, 1), (4800, 64, 4)):
        x, res, dy, dr = (rounded(rng, (rows, D), "bf16").cuda() for _ in range(4))
        w, b = (rounded(rng, (G, D), "f32").cuda() for _ in range(2))
        probs.append((LayerNormBuffers(x, w, b, res=res, groups=G, period=100, with_bwd=True), dy, dr))
    big = max((p[0].ws for p in probs), key=lambda t: t.numel())
    for p in probs:
        p[0].ws = big

    def both(p):
        p[0].forward()
        p[0].backward(p[1], p[2])

    def outs(p):
        return [p[0].y, p[0].r, p[0].dx, p[0].dw, p[0].db]

    eager = []
    for p in probs:
        both(p)
        torch.cuda.synchronize()
        eager.append([t.clone() for t in outs(p)])
    side, graphs = torch.cuda.Stream(), []
    for p in probs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            both(p)
        graphs.append(g)
    for r in range(4):
        for k, p in enumerate(probs):
            for t in outs(p):
                t.fill_(float("nan"))
            graphs[k].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs(p), eager[k])), (r, k)
            both(probs[1 - k])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs(probs[1 - k]), eager[1 - k])), (r, k)


def test_two_streams_at_once():
    """Each with its own workspace; the default stream of the call is the current one."""
    import torch
    from chunkwise_weight_recurrence_amd.layer import LayerNormBuffers
    rng = np.random.default_rng(13)
    probs = []
    for rows, D in ((3000, 1000), (20000, 96)):
        x, dy = (rounded(rng, (rows, D), "bf16").cuda() for _ in range(2))
        probs.append((LayerNormBuffers(x, rounded(rng, (1, D), "f32").cuda(), with_bwd=True), dy))
    want = []
    for p, dy in probs:
        p.forward()
        p.backward(dy)
        torch.cuda.synchronize()
        want.append([t.clone() for t in (p.y, p.dx, p.dw, p.db)])
        for t in (p.y, p.dx, p.dw, p.db):
            t.fill_(float("nan"))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in probs]
    for _ in range(5):
        for (p, dy), s in zip(probs, streams):
            with torch.cuda.stream(s):
                p.forward()
                p.backward(dy)
    torch.cuda.synchronize()
    for (p, _), w in zip(probs, want):
        assert all(torch.equal(a, b) for a, b in zip((p.y, p.dx, p.dw, p.db), w))


def test_single_strided_tokens():
    """[B,1,D] views of a wider tensor: the rows' distance is that of the batch axis."""
    import torch
    from chunkwise_weight_recurrence_amd.layer import LayerNormBuffers
    rng = np.random.default_rng(14)
    for Bn, T, D, room in ((7, 4, 64, 200), (3, 2, 33, 47)):
        wide = torch.full((Bn, T, room), float("nan"), dtype=torch.bfloat16, device="cuda")
        x = wide[:, :1, :D]
        x.copy_(rounded(rng, (Bn, 1, D), "bf16"))
        w, dy = rounded(rng, (1, D), "f32").cuda(), rounded(rng, (Bn, 1, D), "bf16").cuda()
        buf = LayerNormBuffers(x, w, with_bwd=True)
        dwide = torch.full_like(wide, 7.0)
        buf.dx = dwide[:, :1, :D]
        buf.forward()
        buf.backward(dy)
        f = ln.forward(f64(x).reshape(Bn, D), f64(w), None, EPS)
        g = ln.backward(f64(x).reshape(Bn, D), f64(w), EPS, f64(dy).reshape(Bn, D))
        assert worst(buf.y.reshape(Bn, D), f["y"], f["e_y"], "bf16") <= 1
        assert worst(buf.dx.reshape(Bn, D), g["dx"], g["e_dx"], "bf16") <= 1 and worst(buf.dw, g["dw"], g["e_dw"], "f32") <= 1
        assert (dwide[:, 1:] == 7.0).all() and (dwide[..., D:] == 7.0).all()


# From 4096 rows a slot on (slots: 256 threads over the lanes of a narrow row, 512 over a wide one's), a slot takes
# several rows at a time: narrow forwards four, others two.  Each case here has more steps than workgroups, so that
# rows loaded ahead are used, and its last step is ragged.
TOGETHER = [("bf16", 150001, 24, 1, 1, 0, True), ("bf16", 70007, 128, 1, 1, 0, False), ("bf16", 40007, 200, 1, 1, 0, True),
            ("bf16", 20003, 300, 1, 1, 0, True), ("bf16", 150001, 5, 1, 1, 0, True), ("f32", 70001, 63, 1, 1, 0, True),
            ("bf16", 17003, 520, 1, 1, 0, True), ("bf16", 8301, 2048, 1, 1, 0, True), ("bf16", 4501, 2560, 1, 1, 0, True),
            ("f32", 17003, 261, 1, 1, 0, False), ("f32", 4501, 2000, 1, 1, 0, True),
            # a weight for each group, rows apart (their residual stream in place)
            ("bf16", 3 * 11 * 4001, 24, 3, 11, 40, True), ("bf16", 4 * 100 * 43, 520, 4, 100, 528, True),
            ("bf16", 3 * 7 * 3301, 128, 3, 7, 144, False), ("bf16", 4 * 43 * 101, 523, 4, 101, 531, False)]


@pytest.mark.parametrize("dtype,rows,D,groups,period,ldx,residual", TOGETHER)
def test_rows_of_a_slot_together(dtype, rows, D, groups, period, ldx, residual):
    """Every row against the oracle.  dy is whole numbers, so db's sums are exact in fp32 whatever their order, and one
    row too many or too few shows; dw's are off by at most the additions that a product passes through."""
    import torch
    rng = np.random.default_rng(15)
    ld = ldx or D
    wide = torch.full((rows, ld), float("nan"), dtype=torch_dtype(dtype), device="cuda")
    x = wide[:, :D]
    x.copy_(rounded(rng, (rows, D), dtype, mean=0.5, std=2.0))
    res = rounded(rng, (rows, D), dtype).cuda() if residual else None
    kept = (x.float() + res.float()).to(x.dtype) if residual else x
    w, b = rounded(rng, (groups, D), "f32", mean=1.0, std=0.3).cuda(), rounded(rng, (groups, D), "f32").cuda()
    dy = torch.from_numpy(rng.integers(-3, 4, (rows, D)).astype(np.float32)).to(x.dtype).cuda()
    dr = rounded(rng, (rows, D), dtype).cuda() if residual else None
    nan = float("nan")
    y = torch.full((rows, D), nan, dtype=x.dtype, device="cuda")
    mean, rstd = (torch.full((rows,), nan, device="cuda") for _ in range(2))
    dw, db = (torch.full((groups, D), nan, device="cuda") for _ in range(2))
    desc = B.make_ln_desc(rows, D, dtype=dtype, groups=groups, period=period, eps=EPS, ldx=ldx)
    back = B.make_ln_desc(rows, D, dtype=dtype, groups=groups, period=period, eps=EPS) if residual else desc
    dwide = torch.full((rows, D if residual else ld), 7.0, dtype=x.dtype, device="cuda")
    dx = dwide[:, :D]
    ws = torch.full((B.ttt_layernorm_workspace_size(back),), 255, dtype=torch.uint8, device="cuda")
    B.ttt_layernorm_fwd(desc, x, res, w, b, y, res, mean, rstd)
    B.ttt_layernorm_bwd(back, res if residual else x, w, mean, rstd, dy, dr, dx, dw, db, ws)
    torch.cuda.synchronize()
    if residual:
        assert torch.equal(res, kept)
    assert (dwide[:, D:] == 7.0).all()
    r = f64(kept)
    f = ln.forward(r, f64(w), f64(b), EPS, groups, period)
    g = ln.backward(r, f64(w), EPS, f64(dy), f64(dr) if residual else None, groups, period)
    errs = dict(y=worst(y, f["y"], f["e_y"], dtype), mean=worst(mean, f["mean"], f["e_mean"], "f32"),
                rstd=worst(rstd, f["rstd"], f["e_rstd"], "f32"), dx=worst(dx, g["dx"], g["e_dx"], dtype))
    # A thread adds at most 18 rows here (as many as its slot has of the workgroup's), the workgroup 32 slots, the
    # reduction 512 / 32 partial rows a thread and then 32 threads' sums; the product itself is rounded once.
    ops = 18 + 32 + 16 + 32 + 1
    at = ln.groups_of(rows, groups, period)
    size, off = (np.zeros((groups, D)) for _ in range(2))
    for k in range(groups):
        size[k] = np.abs(f64(dy)[at == k] * f["n"][at == k]).sum(0)
        off[k] = (np.abs(f64(dy)[at == k]) * f["e_n"][at == k]).sum(0)
    errs["dw"] = worst(dw, g["dw"], off + ops * ln.U * size, "f32")
    assert all(e <= 1.0 for e in errs.values()), errs
    assert np.array_equal(f64(db), g["db"])
