"""The gated linear recurrence and the layer norm that stand around the fast-weight layer: cases, plain forms and 64-bit values.

`own` False computes them with elementary torch operations in 32 bits; `own` True calls the library's entry points.
"""
import math
import random

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # One new token for each of a few running sequences: a recurrent layer in interactive decoding, bound by launch latency.
        dict(name="rec_step_decode", op="rec_step", rows=8, slots=16, D=2048, dtype="bf16", gate="sigmoid", input="convex"),
        # The same with a full serving batch; the rows name their sequences' places in a larger pool of states.
        dict(name="rec_step_batch", op="rec_step", rows=256, slots=320, D=4096, dtype="bf16", gate="log", input="plain"),
        # The repository's tiny shape: one short chain of 64 channels in fp32.
        dict(name="rec_fwd_tiny", op="rec_fwd", B=1, T=1024, D=64, packed=False, dtype="f32", gate="sigmoid", input="convex"),
        # Prefill of ragged prompts packed behind one another, at the model width of the In-Place configuration.
        dict(name="rec_fwd_prompts", op="rec_fwd", B=37, T=30011, D=2560, packed=True, dtype="bf16", gate="log", input="plain"),
        # One long document, where only a split over the time axis fills the chip.
        dict(name="rec_fwd_long", op="rec_fwd", B=1, T=131072, D=2048, packed=False, dtype="bf16", gate="sigmoid", input="convex"),
        # A training step at the headline shape: 4 sequences of 4096 tokens, 16 heads of 128 channels.
        dict(name="rec_train", op="rec_train", B=4, T=4096, D=2048, packed=False, dtype="bf16", gate="sigmoid", input="convex"),
        # Training on packed documents of odd lengths with an odd width, in fp32, each continuing from a state of its own.
        dict(name="rec_train_odd", op="rec_train", B=19, T=9001, D=1001, packed=True, dtype="f32", gate="sigmoid", input="plain"),
        # The norm of a decode step, with the residual added on the way.
        dict(name="ln_fwd_decode", op="ln_fwd", rows=8, D=2560, groups=1, period=1, residual=True, dtype="bf16"),
        # The norm of a whole 32768-token sequence at the In-Place width.
        dict(name="ln_fwd_prefill", op="ln_fwd", rows=32768, D=2560, groups=1, period=1, residual=True, dtype="bf16"),
        # The pre-norm of a training step, with the gradients of its weight and bias over 16384 rows.
        dict(name="ln_train", op="ln_train", rows=16384, D=2048, groups=1, period=1, residual=True, dtype="bf16"),
        # The norm of the fast-weight layer's output [B, H, T, d], each head with a weight of its own.
        dict(name="ln_train_heads", op="ln_train", rows=4 * 16 * 4096, D=128, groups=16, period=4096, residual=False, dtype="bf16"),
        # Odd sizes in fp32.
        dict(name="ln_train_odd", op="ln_train", rows=3001, D=1001, groups=1, period=1, residual=False, dtype="f32"),
    ]


def _spread(rng, low, high):
    """A whole number of low..high, spread evenly over the logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["rec_step", "rec_fwd", "rec_fwd", "rec_train", "rec_train", "ln_fwd", "ln_train", "ln_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    width = rng.choice([8, 8, 2, 1])  # most widths are whole 16-byte pieces, some are not
    if op.startswith("rec"):
        gate, inp = rng.choice(["sigmoid", "log"]), rng.choice(["plain", "convex"])
        D = max(width, _spread(rng, 48, 4500) // width * width)
        if op == "rec_step":
            rows = _spread(rng, 1, 400)
            return dict(op=op, rows=rows, slots=rows + rng.randrange(0, 64), D=D, dtype=dtype, gate=gate, input=inp)
        tokens = _spread(rng, 1, min(60000, 40_000_000 // D))
        if rng.random() < 0.5:
            return dict(op=op, B=_spread(rng, 1, 200), T=tokens, D=D, packed=True, dtype=dtype, gate=gate, input=inp)
        B = _spread(rng, 1, max(1, min(64, tokens)))
        return dict(op=op, B=B, T=max(1, tokens // B), D=D, packed=False, dtype=dtype, gate=gate, input=inp)
    D = max(width, _spread(rng, 32, 20000) // width * width)
    rows = _spread(rng, 1, 60_000_000 // D)
    groups = period = 1
    if rng.random() < 0.3:
        groups = rng.choice([2, 3, 8, 16])
        period = _spread(rng, 1, max(1, rows // groups))
        rows = max(1, rows // (groups * period)) * groups * period
    return dict(op=op, rows=rows, D=D, groups=groups, period=period, residual=rng.random() < 0.5, dtype=dtype)


def _lengths(total, count, rng):
    """`count` lengths that add up to `total`, spread over a wide range; one of them is zero where there are more than four."""
    share = [math.exp(rng.uniform(0.0, 4.0)) for _ in range(count)]
    if count > 4:
        share[rng.randrange(count)] = 0.0
    scale, at, edges = total / sum(share), 0.0, [0]
    for s in share:
        at += s * scale
        edges.append(min(total, int(round(at))))
    edges[-1] = total
    return edges


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, mean=0.0, std=1.0, dtype=torch.float32):
        return torch.empty(shape, device=DEVICE, dtype=torch.float32).normal_(mean, std, generator=g).to(dtype)

    s = dict(case=case)
    D = case["D"]
    if case["op"].startswith("rec"):
        B = case["B"] if "B" in case else case["rows"]
        if case["op"] == "rec_step":
            shape = (B, D)
            s["h"] = normal(case["slots"], D, std=0.5)
            s["slots"] = torch.randperm(case["slots"], generator=g, device=DEVICE)[:B].to(torch.int32)
        else:
            shape = (case["T"], D) if case["packed"] else (B, case["T"], D)
            s["h0"] = normal(B, D, std=0.5)
            s["starts"] = None
            if case["packed"]:
                s["edges"] = _lengths(case["T"], B, random.Random(seed))
                s["starts"] = torch.tensor(s["edges"], dtype=torch.int32, device=DEVICE)
        s["x"] = normal(*shape, dtype=dt)
        # decays as the fast-weight layer's vector decay has them: a = sigmoid(z), z ~ N(4, 1)
        z = normal(*shape, mean=4.0)
        s["gate"] = (z if case["gate"] == "sigmoid" else torch.nn.functional.logsigmoid(z)).to(dt)
        if case["op"] == "rec_train":
            s["d_o"] = normal(*shape, dtype=dt)
            s["d_hfinal"] = normal(B, D)
        return s
    rows = case["rows"]
    # rows with means and scales of their own, as a residual stream has
    s["x"] = (normal(rows, D) * normal(rows, 1).exp() + normal(rows, 1)).to(dt)
    s["res"] = normal(rows, D, dtype=dt) if case["residual"] else None
    s["w"] = 1.0 + normal(case["groups"], D, std=0.2)
    s["b"] = normal(case["groups"], D, std=0.2)
    if case["op"] == "ln_train":
        s["dy"] = normal(rows, D, dtype=dt)
        s["dr"] = normal(rows, D, dtype=dt) if case["residual"] else None
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return _own_recurrence(state) if op.startswith("rec") else _own_norm(state)
    if op == "rec_step":
        return _plain_step(state)
    return _plain_recurrence(state) if op.startswith("rec") else _plain_norm(state)


# The framework's calls.


def _own_recurrence(state):
    import chunkwise_weight_recurrence_amd as F
    c = state["case"]
    plan = state.get("plan")
    if plan is None:  # the descriptor and the buffers that a program keeps from call to call
        plan = state["plan"] = {}
        f32 = dict(dtype=torch.float32, device=DEVICE)
        plan["o"] = torch.empty_like(state["x"])
        if c["op"] == "rec_step":
            plan["desc"] = F.make_rec_desc(c["rows"], 1, c["D"], dtype=c["dtype"], gate=c["gate"], input=c["input"])
            plan["h"] = state["h"].clone()
        else:
            desc = plan["desc"] = F.make_rec_desc(c["B"], c["T"], c["D"], dtype=c["dtype"], gate=c["gate"], input=c["input"], packed=c["packed"])
            plan["h_final"] = torch.empty((c["B"], c["D"]), **f32)
            size = F.ttt_recurrence_workspace_size(desc, F.ENTRY_FWD)
            plan["saved"] = None
            if c["op"] == "rec_train":
                size = max(size, F.ttt_recurrence_workspace_size(desc, F.ENTRY_BWD))
                plan["saved"] = torch.empty(F.ttt_recurrence_saved_size(desc), dtype=torch.uint8, device=DEVICE)
                plan["dx"], plan["dgate"] = torch.empty_like(state["x"]), torch.empty_like(state["x"])
                plan["dh0"] = torch.empty((c["B"], c["D"]), **f32)
            plan["ws"] = torch.empty(size, dtype=torch.uint8, device=DEVICE)
    p = plan
    if c["op"] == "rec_step":
        # the state moves on in place; each pass begins from the same one
        p["h"].copy_(state["h"])
        F.ttt_recurrence_step(p["desc"], state["x"], state["gate"], state["slots"], p["h"], p["o"])
        return {"o": p["o"], "h": p["h"]}
    F.ttt_recurrence_fwd(p["desc"], state["x"], state["gate"], state["h0"], state["starts"], p["o"], p["h_final"], p["saved"], p["ws"])
    out = {"o": p["o"], "h_final": p["h_final"]}
    if c["op"] == "rec_train":
        F.ttt_recurrence_bwd(p["desc"], state["x"], state["gate"], state["h0"], state["starts"], p["saved"], state["d_o"], state["d_hfinal"],
                             p["dx"], p["dgate"], p["dh0"], p["ws"])
        out.update(dx=p["dx"], dgate=p["dgate"], dh0=p["dh0"])
    return out


def _own_norm(state):
    import chunkwise_weight_recurrence_amd as F
    c = state["case"]
    plan = state.get("plan")
    if plan is None:
        plan = state["plan"] = {}
        rows, D, x = c["rows"], c["D"], state["x"]
        desc = plan["desc"] = F.make_ln_desc(rows, D, dtype=c["dtype"], groups=c["groups"], period=c["period"], eps=EPS)
        plan["y"] = torch.empty_like(x)
        plan["r"] = torch.empty_like(x) if c["residual"] else None
        plan["mean"] = plan["rstd"] = None
        if c["op"] == "ln_train":
            plan["mean"] = torch.empty(rows, dtype=torch.float32, device=DEVICE)
            plan["rstd"] = torch.empty(rows, dtype=torch.float32, device=DEVICE)
            plan["dx"], plan["dw"], plan["db"] = torch.empty_like(x), torch.empty_like(state["w"]), torch.empty_like(state["b"])
            plan["ws"] = torch.empty(F.ttt_layernorm_workspace_size(desc), dtype=torch.uint8, device=DEVICE)
    p = plan
    F.ttt_layernorm_fwd(p["desc"], state["x"], state["res"], state["w"], state["b"], p["y"], p["r"], p["mean"], p["rstd"])
    out = {"y": p["y"]}
    if c["residual"]:
        out["r"] = p["r"]
    if c["op"] == "ln_train":
        F.ttt_layernorm_bwd(p["desc"], p["r"] if c["residual"] else state["x"], state["w"], p["mean"], p["rstd"], state["dy"], state["dr"],
                            p["dx"], p["dw"], p["db"], p["ws"])
        out.update(dx=p["dx"], dw=p["dw"], db=p["db"])
    return out


# The plain forms.


def _coefficients(state):
    """a, da/dgate and the input's factor in 32 bits: h_t = a_t h_{t-1} + f_t x_t."""
    c = state["case"]
    g = state["gate"].float()
    if c["gate"] == "sigmoid":
        a = 1 / (1 + torch.exp(-g))
        rest = 1 / (1 + torch.exp(g))
        da = a * rest
    else:
        a = torch.exp(g)
        rest = -torch.expm1(g)
        da = a
    return a, da, rest if c["input"] == "convex" else None


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along axis 0, h_{-1} = 0, by doubling; a and b are used up."""
    step = 1
    while step < a.shape[0]:
        b[step:] += a[step:] * b[:-step].clone()
        a[step:] *= a[:-step].clone()
        step *= 2
    return b


def _plain_recurrence(state):
    c = state["case"]
    B, T, D = c["B"], c["T"], c["D"]
    n = T if c["packed"] else B * T
    x = state["x"].float().reshape(n, D)
    a, da, f = (v.reshape(n, D) if v is not None else None for v in _coefficients(state))
    u = x if f is None else f * x
    starts = state["starts"].long() if c["packed"] else torch.arange(0, n + 1, T, device=x.device)
    kept = (starts[1:] > starts[:-1]).nonzero()[:, 0]  # the sequences that have a token
    first, last = starts[:-1][kept], starts[1:][kept] - 1
    coef, b = a.clone(), u.clone()
    b[first] += a[first] * state["h0"][kept]
    coef[first] = 0
    h = _scan(coef, b)
    h_final = state["h0"].clone()
    h_final[kept] = h[last]
    out = {"o": h.to(state["x"].dtype).reshape(state["x"].shape), "h_final": h_final}
    if c["op"] == "rec_train":
        # dh_t = d_o_t + a_{t+1} dh_{t+1}, the same scan from the end
        coef = torch.cat([a[1:], a[:1]])
        coef[last] = 0
        b = state["d_o"].float().reshape(n, D)
        b = b.clone() if b is state["d_o"] or b.data_ptr() == state["d_o"].data_ptr() else b
        b[last] += state["d_hfinal"][kept]
        dh = _scan(coef.flip(0), b.flip(0)).flip(0)
        before = torch.cat([h[:1], h[:-1]])
        before[first] = state["h0"][kept]
        dx = dh if f is None else dh * f
        dgate = dh * da * (before if f is None else before - x)
        dh0 = state["d_hfinal"].clone()
        dh0[kept] = a[first] * dh[first]
        shape, dt = state["x"].shape, state["x"].dtype
        out.update(dx=dx.to(dt).reshape(shape), dgate=dgate.to(dt).reshape(shape), dh0=dh0)
    return out


def _plain_step(state):
    a, _, f = _coefficients(state)
    x = state["x"].float()
    at = state["slots"].long()
    new = a * state["h"][at] + (x if f is None else f * x)
    h = state["h"].clone()
    h[at] = new
    return {"o": new.to(state["x"].dtype), "h": h}


def _plain_norm(state):
    c = state["case"]
    rows, D, G = c["rows"], c["D"], c["groups"]
    dt = state["x"].dtype
    x = state["x"].float()
    out = {}
    if c["residual"]:
        # the stream that the next layer reads is what is normalised
        out["r"] = (x + state["res"].float()).to(dt)
        x = out["r"].float()
    mean = x.mean(1, keepdim=True)
    xc = x - mean
    rstd = 1 / torch.sqrt((xc * xc).mean(1, keepdim=True) + EPS)
    hat = xc * rstd
    heads = (rows // (G * c["period"]), G, c["period"], D) if G > 1 else (1, 1, rows, D)
    w, b = state["w"].view(1, G, 1, D), state["b"].view(1, G, 1, D)
    out["y"] = (hat.view(heads) * w + b).to(dt).view(rows, D)
    if c["op"] == "ln_train":
        dy = state["dy"].float()
        wdy = (dy.view(heads) * w).view(rows, D)
        dx = rstd * (wdy - wdy.mean(1, keepdim=True) - hat * (wdy * hat).mean(1, keepdim=True))
        if c["residual"]:
            dx = dx + state["dr"].float()
        out["dx"] = dx.to(dt)
        out["dw"] = (dy * hat).view(heads).sum((0, 2))
        out["db"] = dy.view(heads).sum((0, 2))
    return out


def work(case):
    """Each call's inputs read once and its outputs written once (a training step is a forward call and, later, a backward call)."""
    D, e = case["D"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rec_step":
        # the pool's other states pass through untouched; the copy that resets the pool between passes is part of the pass
        n = case["rows"] * D
        return {"bytes": n * (3 * e + 8) + 8 * case["slots"] * D, "flops": 8 * n}
    if case["op"].startswith("rec"):
        n = (case["T"] if case["packed"] else case["B"] * case["T"]) * D
        state = 4 * case["B"] * D
        if case["op"] == "rec_fwd":
            return {"bytes": 3 * e * n + 2 * state, "flops": 8 * n}
        return {"bytes": 8 * e * n + 5 * state, "flops": 24 * n}
    n, r = case["rows"] * D, case["residual"]
    weights = 8 * case["groups"] * D
    if case["op"] == "ln_fwd":
        return {"bytes": n * e * (4 if r else 2) + weights, "flops": 8 * n}
    return {"bytes": n * e * (4 + 4 if r else 2 + 3) + 16 * case["rows"] + 2.5 * weights, "flops": 24 * n}


def exact(case, seed):
    """The definitions, token by token and row by row, in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "rec_step":
        return _exact_step(s)
    if case["op"].startswith("rec"):
        steps = case["T"] * (2 if case["op"] == "rec_train" else 1)
        return _exact_recurrence(s) if steps <= 140_000 else None
    return _exact_norm(s)


def _decay64(s):
    g = s["gate"].double()
    a = torch.sigmoid(g) if s["case"]["gate"] == "sigmoid" else g.exp()
    keep = 1 if s["case"]["input"] == "plain" else (torch.sigmoid(-g) if s["case"]["gate"] == "sigmoid" else -torch.expm1(g))
    return a, keep


def _exact_step(s):
    a, keep = _decay64(s)
    h = s["h"].double()
    at = s["slots"].long()
    h[at] = a * h[at] + keep * s["x"].double()
    return {"o": h[at], "h": h}


def _exact_recurrence(s):
    c = s["case"]
    a, keep = _decay64(s)
    x = s["x"].double()
    u = keep * x
    train = c["op"] == "rec_train"
    o = torch.empty_like(u)
    final = s["h0"].double()
    # each piece: the index of its states, and views with the time axis in front
    if c["packed"]:
        pieces = [(i, slice(p, q)) for i, (p, q) in enumerate(zip(s["edges"], s["edges"][1:])) if q > p]
        view = lambda v, at: v[at]  # noqa: E731
    else:
        pieces = [(slice(None), None)]
        view = lambda v, at: v.transpose(0, 1)  # noqa: E731
    grads = {}
    if train:
        d_o = s["d_o"].double()
        dx, dgate = torch.empty_like(u), torch.empty_like(u)
        dh0 = s["d_hfinal"].double()
        slope = a if c["gate"] == "log" else a * torch.sigmoid(-s["gate"].double())
        grads = {"dx": dx, "dgate": dgate, "dh0": dh0}
    for i, at in pieces:
        av, uv, ov = view(a, at), view(u, at), view(o, at)
        h = final[i].clone()
        for t in range(av.shape[0]):
            h = torch.addcmul(uv[t], av[t], h)
            ov[t] = h
        final[i] = h
        if train:
            dv = view(d_o, at)
            dh = torch.empty_like(dv)
            e = dh0[i].clone()
            for t in range(av.shape[0] - 1, -1, -1):
                e = dv[t] + e
                dh[t] = e
                e = e * av[t]
            dh0[i] = e
            before = torch.cat([s["h0"][i].double().reshape(1, *h.shape), ov[:-1]])
            view(dx, at)[:] = dh * (view(keep, at) if torch.is_tensor(keep) else 1)
            view(dgate, at)[:] = dh * view(slope, at) * (before - (view(x, at) if c["input"] == "convex" else 0))
    return {"o": o, "h_final": final, **grads}


def _exact_norm(s):
    c = s["case"]
    out = {}
    x = s["x"].double()
    if c["residual"]:
        r = (s["x"].double() + s["res"].double())
        out["r"] = r
        x = r.to(s["x"].dtype).double()  # the norm is of the rows as they are kept
    mean = x.mean(1, keepdim=True)
    var = ((x - mean) ** 2).mean(1, keepdim=True)
    hat = (x - mean) / (var + EPS).sqrt()
    group = (torch.arange(c["rows"], device=x.device) // c["period"]) % c["groups"]
    w = s["w"].double()[group]
    out["y"] = hat * w + s["b"].double()[group]
    if c["op"] == "ln_train":
        dy = s["dy"].double()
        wdy = w * dy
        dx = (wdy - wdy.mean(1, keepdim=True) - hat * (wdy * hat).mean(1, keepdim=True)) / (var + EPS).sqrt()
        out["dx"] = dx + s["dr"].double() if c["residual"] else dx
        zero = torch.zeros_like(s["w"], dtype=torch.float64)
        out["dw"] = zero.index_add(0, group, dy * hat)
        out["db"] = zero.index_add(0, group, dy)
    return out
