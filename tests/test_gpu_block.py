"""The operators together, as a model uses them: residual norm -> recurrence -> norm per head,
and the fast-weight layer with a norm per head behind it, forward and backward."""
import numpy as np
import pytest

from chunkwise_weight_recurrence_amd import workloads as wl
from oracle import layernorm_oracle as ln
from oracle import recurrence_oracle as rec
from tests.block_utils import f64, rounded
from tests.parity_utils import compare, rel_err, small_cfg

pytestmark = pytest.mark.gpu

EPS = 1e-5
# max |gpu - fp64| / max |fp64|, as for the fast-weight layer.  fp32: each of the six
# passes adds at most about 100 roundings of 2^-24 and passes on what it gets with a
# gain below 3 (the norms' 1 / deviation and weights): 6 * 100 * 2^-24 * 3 = 1.1e-4
# of the largest value at the very worst.
# bf16: every operator rounds its output (2^-8 / 2 of the value), the norms' gains as above: below 2e-2.
TOL = {"f32": 1.1e-4, "bf16": 2e-2}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("packed", [False, True])
def test_recurrent_block(dtype, packed):
    import torch
    from chunkwise_weight_recurrence_amd.layer import LayerNormBuffers, RecurrenceBuffers
    Bn, T, H, d = 2, 201, 4, 24
    D, n = H * d, 2 * 201
    starts = [0, 150, 150, 397, 402] if packed else rec.dense_starts(Bn, T).tolist()
    rng = np.random.default_rng(0)
    x, res, gate = rounded(rng, (n, D), dtype), rounded(rng, (n, D), dtype), rounded(rng, (n, D), dtype, mean=2.0)
    w1, b1 = rounded(rng, (1, D), "f32", mean=1.0, std=0.2), rounded(rng, (1, D), "f32", std=0.2)
    w2, b2 = rounded(rng, (H, d), "f32", mean=1.0, std=0.2), rounded(rng, (H, d), "f32", std=0.2)
    dy, dr = rounded(rng, (n, D), dtype), rounded(rng, (n, D), dtype)
    shape = (n, D) if packed else (Bn, T, D)
    norm1 = LayerNormBuffers(x.cuda().view(shape), w1.cuda(), b1.cuda(), res=res.cuda().view(shape), with_bwd=True)
    st = torch.tensor(starts, dtype=torch.int32).cuda() if packed else None
    mix = RecurrenceBuffers(norm1.y, gate.cuda().view(shape), seq_starts=st, with_bwd=True)
    norm2 = LayerNormBuffers(mix.o.view(n * H, d), w2.cuda(), b2.cuda(), groups=H, period=1, with_bwd=True)
    norm1.forward()
    mix.forward()
    norm2.forward()
    norm2.backward(dy.cuda().view(n * H, d))
    mix.backward(norm2.dx.view(shape))
    norm1.backward(mix.dx, dr.cuda().view(shape))
    torch.cuda.synchronize()
    got = dict(y=norm2.y, r=norm1.r, dx=norm1.dx, dgate=mix.dgate, dw1=norm1.dw, db1=norm1.db, dw2=norm2.dw, db2=norm2.db)

    r = f64(x) + f64(res)
    f1 = ln.forward(r, f64(w1), f64(b1), EPS)
    o, _, _, _ = rec.forward(f1["y"], f64(gate), starts, "sigmoid", "convex")
    f2 = ln.forward(o.reshape(n * H, d), f64(w2), f64(b2), EPS, H, 1)
    g2 = ln.backward(o.reshape(n * H, d), f64(w2), EPS, f64(dy).reshape(n * H, d), None, H, 1)
    gm = rec.backward(f1["y"], f64(gate), starts, "sigmoid", "convex", g2["dx"].reshape(n, D))
    g1 = ln.backward(r, f64(w1), EPS, gm["dx"], f64(dr))
    want = dict(y=f2["y"], r=r, dx=g1["dx"], dgate=gm["dgate"], dw1=g1["dw"], db1=g1["db"], dw2=g2["dw"], db2=g2["db"])
    errs = {k: rel_err(f64(got[k]).reshape(want[k].shape), want[k]) for k in want}
    print(f"[block] {dtype} packed={packed} " + " ".join(f"{k}={v:.1e}" for k, v in errs.items()), flush=True)
    assert all(e <= TOL[dtype] for e in errs.values()), errs


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_fast_weight_layer_with_a_norm_per_head(dtype):
    import torch
    from chunkwise_weight_recurrence_amd.layer import LayerNormBuffers, TTTLayerBuffers
    from oracle import chunk_backward, chunk_forward
    cfg = small_cfg(dtype, "mse", "none", "scalar", B=2, H=3, T=200, b=-4.0)
    inp = wl.make_ttt_inputs(cfg)
    rng = np.random.default_rng(1)
    H, T, d = 3, 200, cfg["dv"]
    w, b = rounded(rng, (H, d), "f32", mean=1.0, std=0.2), rounded(rng, (H, d), "f32", std=0.2)
    dy = rounded(rng, (2 * H * T, d), dtype)
    layer = TTTLayerBuffers(inp)
    layer.forward()
    norm = LayerNormBuffers(layer.o, w.cuda(), b.cuda(), groups=H, period=T, with_bwd=True)
    norm.forward()
    norm.backward(dy.cuda())
    layer.d_o = norm.dx
    layer.backward()
    torch.cuda.synchronize()
    # the norm's part against the fp64 norm of the layer's own output, the layer's against the oracle on the norm's gradient
    o = f64(layer.o).reshape(-1, d)
    f, g = ln.forward(o, f64(w), f64(b), EPS, H, T), ln.backward(o, f64(w), EPS, f64(dy), None, H, T)
    kw = wl.oracle_kwargs(inp)
    O, _, _ = chunk_forward(inp["q"], inp["k"], inp["v"], inp["beta"], cfg["b"], cfg["C"], return_ckpt=True, **kw)
    gl = chunk_backward(inp["q"], inp["k"], inp["v"], inp["beta"], cfg["b"], cfg["C"], f64(norm.dx), **kw)
    got = dict(O=f64(layer.o), y=f64(norm.y).reshape(-1, d), d_o=f64(norm.dx).reshape(-1, d), dw=f64(norm.dw), db=f64(norm.db),
               dq=f64(layer.dq), dk=f64(layer.dk), dv=f64(layer.dv))
    want = dict(O=O, y=f["y"], d_o=g["dx"], dw=g["dw"], db=g["db"], dq=gl["dq"], dk=gl["dk"], dv=gl["dv"])
    errs, bad = compare(got, want, dtype)
    assert not bad, errs
