"""The gated delta rule and the norm and rotation of its queries and keys: cases, plain forms and 64-bit values.

`own` False computes them with elementary torch operations in 32 bits; `own` True calls the library's entry points.
"""
import math
import random

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
CHUNK = 64  # of the plain form


def listed():
    return [
        # One new token for each of a few running sequences: interactive decoding, bound by launch latency and one pass over the states.
        dict(name="delta_step_decode", op="delta_step", rows=8, slots=16, H=16, Hk=16, dk=128, dv=128, dtype="bf16", gate="sigmoid"),
        # A full serving batch with two value heads on each key head; the rows name their places in a larger pool of states.
        dict(name="delta_step_batch", op="delta_step", rows=256, slots=320, H=16, Hk=8, dk=128, dv=128, dtype="bf16", gate="log"),
        # The repository's tiny shape: one short chain of 64 channels in fp32.
        dict(name="delta_fwd_tiny", op="delta_fwd", B=1, T=1024, H=1, Hk=1, dk=64, dv=64, packed=False, fused=False, dtype="f32", gate="sigmoid"),
        # Prefill of ragged prompts packed behind one another, at the model width of the In-Place configuration (20 heads of 128).
        dict(name="delta_fwd_prompts", op="delta_fwd", B=37, T=30011, H=20, Hk=20, dk=128, dv=128, packed=True, fused=True, dtype="bf16", gate="log"),
        # One long document, where only a split over the time axis fills the chip.
        dict(name="delta_fwd_long", op="delta_fwd", B=1, T=131072, H=16, Hk=16, dk=128, dv=128, packed=False, fused=False, dtype="bf16", gate="sigmoid"),
        # A training step at the headline shape: 4 sequences of 4096 tokens, 16 heads of 128 channels.
        dict(name="delta_train", op="delta_train", B=4, T=4096, H=16, Hk=16, dk=128, dv=128, packed=False, fused=True, dtype="bf16", gate="sigmoid"),
        # Training on packed documents of odd lengths, odd head widths and shared key heads, in fp32.
        dict(name="delta_train_odd", op="delta_train", B=19, T=9001, H=6, Hk=3, dk=50, dv=37, packed=True, fused=False, dtype="f32", gate="log"),
        # The norm and rotation of a decode step, at positions deep in a long context whose frequencies are scaled.
        dict(name="qk_fwd_decode", op="qk_fwd", tokens=8, Hq=16, Hk=16, d=128, rot=128, pairing="half", norm="rms", weight=True, far=True, dtype="bf16"),
        # The same for a whole 32768-token sequence at the In-Place width, the projections in one buffer.
        dict(name="qk_fwd_prefill", op="qk_fwd", tokens=32768, Hq=20, Hk=20, d=128, rot=128, pairing="half", norm="rms", weight=True, far=False, dtype="bf16"),
        # A training step: unit queries and keys for the delta rule, half of each head rotated.
        dict(name="qk_train", op="qk_train", tokens=16384, Hq=16, Hk=16, d=128, rot=64, pairing="interleaved", norm="l2", weight=False, far=False, dtype="bf16"),
        # Training with the norm's weights and fewer key heads than query heads.
        dict(name="qk_train_weights", op="qk_train", tokens=16384, Hq=16, Hk=4, d=64, rot=64, pairing="half", norm="rms", weight=True, far=False, dtype="bf16"),
        # Odd sizes in fp32.
        dict(name="qk_train_odd", op="qk_train", tokens=3001, Hq=5, Hk=1, d=70, rot=34, pairing="interleaved", norm="rms", weight=True, far=True, dtype="f32"),
    ]


def _spread(rng, low, high):
    """A whole number of low..high, spread evenly over the logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["delta_step", "delta_fwd", "delta_fwd", "delta_train", "delta_train", "qk_fwd", "qk_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("delta"):
        def width():
            return rng.choice([64, 64, 128, 128, 256, 96, _spread(rng, 8, 256), _spread(rng, 8, 256)])
        dk, dv, Hk = width(), width(), _spread(rng, 1, 16)
        H = Hk * rng.choice([1, 1, 2, 3])
        gate = rng.choice(["sigmoid", "log"])
        if op == "delta_step":
            rows = _spread(rng, 1, max(1, min(400, 60_000_000 // (H * dk * dv))))
            return dict(op=op, rows=rows, slots=rows + rng.randrange(0, 64), H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype, gate=gate)
        # up to a quarter of the longest case's work in bf16, less in fp32 and with gradients
        most = 60_000_000 // (H * max(dk, dv)) // (4 if dtype == "f32" else 1) // (4 if op == "delta_train" else 1)
        tokens = _spread(rng, 1, max(16, min(60000, most)))
        if rng.random() < 0.5:
            return dict(op=op, B=_spread(rng, 1, 100), T=tokens, H=H, Hk=Hk, dk=dk, dv=dv, packed=True, fused=rng.random() < 0.5, dtype=dtype, gate=gate)
        B = _spread(rng, 1, max(1, min(32, tokens)))
        return dict(op=op, B=B, T=max(1, tokens // B), H=H, Hk=Hk, dk=dk, dv=dv, packed=False, fused=rng.random() < 0.5, dtype=dtype, gate=gate)
    d = rng.choice([64, 64, 128, 128, 256, 80, 2 * _spread(rng, 4, 128), 2 * _spread(rng, 4, 128)])
    Hk = _spread(rng, 1, 20)
    Hq = Hk * rng.choice([1, 1, 2, 4])
    rot = rng.choice([d, d, d // 4 * 2, 0, 2 * rng.randrange(0, d // 2 + 1)])
    return dict(op=op, tokens=_spread(rng, 1, max(1, min(60000, 60_000_000 // ((Hq + Hk) * d)))), Hq=Hq, Hk=Hk, d=d, rot=rot,
                pairing=rng.choice(["half", "interleaved"]), norm=rng.choice(["rms", "l2", "none"]), weight=rng.random() < 0.5,
                far=rng.random() < 0.5, dtype=dtype)


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

    def split(n, fused, *parts):
        """Rows of [heads, d] tensors, as slices of one projection's output where `fused`."""
        if not fused:
            return [p.to(dt) for p in parts]
        whole = torch.cat([p.reshape(n, -1) for p in parts], 1).to(dt)
        out, at = [], 0
        for p in parts:
            w = p.shape[1] * p.shape[2]
            out.append(whole[:, at:at + w].view(p.shape))
            at += w
        return out

    s = dict(case=case)
    if case["op"].startswith("qk"):
        n, Hq, Hk, d = case["tokens"], case["Hq"], case["Hk"], case["d"]
        heads = lambda H: normal(n, H, d) * normal(n, H, 1, std=0.5).exp()  # noqa: E731  heads with scales of their own
        s["q"], s["k"] = split(n, True, heads(Hq), heads(Hk))
        s["wq"] = 1.0 + normal(d, std=0.2) if case["weight"] else None
        s["wk"] = 1.0 + normal(d, std=0.2) if case["weight"] else None
        if case["far"]:  # frequencies stretched for a context of a million tokens
            s["pos"] = torch.randint(0, 1_000_000, (n,), generator=g, device=DEVICE).to(torch.int32)
            base, stretch = 5e5, 8.0
        else:
            s["pos"] = torch.arange(n, device=DEVICE, dtype=torch.int32)
            base, stretch = 1e4, 1.0
        half = case["rot"] // 2
        s["inv_freq"] = (base ** (-torch.arange(half, device=DEVICE, dtype=torch.float64) / max(1, half)) / stretch).float()
        if case["op"] == "qk_train":
            s["dyq"], s["dyk"] = normal(n, Hq, d, dtype=dt), normal(n, Hk, d, dtype=dt)
        return s
    H, Hk, dk, dv = case["H"], case["Hk"], case["dk"], case["dv"]
    step = case["op"] == "delta_step"
    B = case["rows"] if step else case["B"]
    n = B if step else case["T"] if case["packed"] else B * case["T"]
    unit = lambda: torch.nn.functional.normalize(normal(n, Hk, dk), dim=-1)  # noqa: E731  as the norm leaves them
    s["q"], s["k"], s["v"] = split(n, step or case["fused"], unit(), unit(), normal(n, H, dv))
    # decays as the fast-weight layer's have them: a = sigmoid(z), z ~ N(4, 1)
    z = normal(n, H, mean=4.0)
    s["gate"] = (z if case["gate"] == "sigmoid" else torch.nn.functional.logsigmoid(z)).to(dt)
    s["beta"] = normal(n, H, dtype=dt)
    if step:
        s["s"] = normal(case["slots"], H, dk, dv, std=0.3)
        s["slots"] = torch.randperm(case["slots"], generator=g, device=DEVICE)[:B].to(torch.int32)
        return s
    s["s0"] = normal(B, H, dk, dv, std=0.3)
    s["edges"] = _lengths(n, B, random.Random(seed)) if case["packed"] else list(range(0, n + 1, case["T"]))
    s["starts"] = torch.tensor(s["edges"], dtype=torch.int32, device=DEVICE) if case["packed"] else None
    if case["op"] == "delta_train":
        s["d_o"] = normal(n, H, dv, dtype=dt)
        s["d_sfinal"] = normal(B, H, dk, dv, std=0.3)
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return _own_qk(state) if op.startswith("qk") else _own_delta(state)
    if op == "delta_step":
        return _plain_step(state)
    return _plain_qk(state) if op.startswith("qk") else _plain_delta(state)


# The framework's calls.


def _own_delta(state):
    import chunkwise_weight_recurrence_amd as F
    c = state["case"]
    step = c["op"] == "delta_step"
    plan = state.get("plan")
    if plan is None:  # the descriptor and the buffers that a program keeps from call to call
        plan = state["plan"] = {}
        f32 = dict(dtype=torch.float32, device=DEVICE)
        B, T = (c["rows"], 1) if step else (c["B"], c["T"])
        desc = plan["desc"] = F.make_delta_desc(B, T, c["H"], c["dk"], c["dv"], Hk=c["Hk"], dtype=c["dtype"], gate=c["gate"],
                                                packed=not step and c["packed"], scale=c["dk"] ** -0.5,
                                                ldq=state["q"].stride(0), ldk=state["k"].stride(0), ldv=state["v"].stride(0))
        plan["o"] = torch.empty(state["v"].shape, dtype=state["v"].dtype, device=DEVICE)
        if step:
            plan["s"] = state["s"].clone()
        else:
            plan["s_final"] = torch.empty((B, c["H"], c["dk"], c["dv"]), **f32)
            size = F.ttt_delta_workspace_size(desc, F.ENTRY_FWD)
            plan["saved"] = None
            if c["op"] == "delta_train":
                size = max(size, F.ttt_delta_workspace_size(desc, F.ENTRY_BWD))
                plan["saved"] = torch.empty(F.ttt_delta_saved_size(desc), dtype=torch.uint8, device=DEVICE)
                for name in "qkv":
                    x = state[name]
                    plan["d" + name] = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=DEVICE)
                plan["dgate"], plan["dbeta"] = torch.empty_like(state["gate"]), torch.empty_like(state["beta"])
                plan["ds0"] = torch.empty_like(state["s0"])
            plan["ws"] = torch.empty(size, dtype=torch.uint8, device=DEVICE)
    p, s = plan, state
    if step:
        # the new states go beside the old ones, as where a token may be taken back
        F.ttt_delta_step(p["desc"], s["q"], s["k"], s["v"], s["gate"], s["beta"], s["slots"], s["s"], p["s"], p["o"])
        return {"o": p["o"], "s": p["s"]}
    F.ttt_delta_fwd(p["desc"], s["q"], s["k"], s["v"], s["gate"], s["beta"], s["s0"], s["starts"], p["o"], p["s_final"], p["saved"], p["ws"])
    out = {"o": p["o"], "s_final": p["s_final"]}
    if c["op"] == "delta_train":
        F.ttt_delta_bwd(p["desc"], s["q"], s["k"], s["v"], s["gate"], s["beta"], s["starts"], p["saved"], s["d_o"], s["d_sfinal"],
                        p["dq"], p["dk"], p["dv"], p["dgate"], p["dbeta"], p["ds0"], p["ws"])
        out.update({x: p[x] for x in ("dq", "dk", "dv", "dgate", "dbeta", "ds0")})
    return out


def _own_qk(state):
    import chunkwise_weight_recurrence_amd as F
    c = state["case"]
    plan = state.get("plan")
    if plan is None:
        plan = state["plan"] = {}
        q, k = state["q"], state["k"]
        desc = plan["desc"] = F.make_qknorm_desc(c["tokens"], c["Hq"], c["Hk"], c["d"], rot=c["rot"], pairing=c["pairing"], norm=c["norm"],
                                                 dtype=c["dtype"], eps=EPS, ldq=q.stride(0), ldk=k.stride(0))
        plan["yq"], plan["yk"] = (torch.empty(x.shape, dtype=x.dtype, device=DEVICE) for x in (q, k))
        if c["op"] == "qk_train":
            plan["dq"], plan["dk"] = (torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=DEVICE) for x in (q, k))
            plan["dwq"], plan["dwk"] = (torch.empty_like(state[x]) if c["weight"] else None for x in ("wq", "wk"))
            plan["ws"] = torch.empty(F.ttt_qknorm_workspace_size(desc), dtype=torch.uint8, device=DEVICE)
    p, s = plan, state
    F.ttt_qknorm_fwd(p["desc"], s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["inv_freq"], p["yq"], p["yk"])
    out = {"yq": p["yq"], "yk": p["yk"]}
    if c["op"] == "qk_train":
        F.ttt_qknorm_bwd(p["desc"], s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["inv_freq"], s["dyq"], s["dyk"], p["dq"], p["dk"],
                         p["dwq"], p["dwk"], p["ws"])
        out.update(dq=p["dq"], dk=p["dk"])
        if c["weight"]:
            out.update(dwq=p["dwq"], dwk=p["dwk"])
    return out


# The plain forms.


def _gate_and_rate(state):
    """log a, d log a / d gate, eta, and d eta / d beta over eta in 32 bits."""
    z, b = state["gate"].float(), state["beta"].float()
    eta = 1 / (1 + torch.exp(-b))
    if state["case"]["gate"] == "log":
        return z, torch.ones_like(z), eta, 1 / (1 + torch.exp(b))
    return torch.clamp(z, max=0) - torch.log1p(torch.exp(-z.abs())), 1 / (1 + torch.exp(z)), eta, 1 / (1 + torch.exp(b))


def _plain_step(state):
    c = state["case"]
    g, _, eta, _ = _gate_and_rate(state)
    share = c["H"] // c["Hk"]
    q, k = (state[x].float().repeat_interleave(share, 1) for x in "qk")
    at = state["slots"].long()
    s = state["s"].clone()
    new = s[at] * torch.exp(g)[..., None, None]
    e = state["v"].float() - (new * k[..., None]).sum(2)
    new = new + k[..., None] * (eta[..., None] * e)[:, :, None]
    s[at] = new
    o = (new * q[..., None]).sum(2) * c["dk"] ** -0.5
    return {"o": o.to(state["v"].dtype), "s": s}


def _plain_delta(state):
    """By chunks of tokens: with G the sum of log a and R_ij = exp(G_i - G_j), u = eta (v - S'^T k) of a chunk solves
    u_i + eta_i sum_{j<i} R_ij (k_i.k_j) u_j = eta_i (v_i - e^{G_i} S^T k_i)."""
    c = state["case"]
    H, dk, dv, C = c["H"], c["dk"], c["dv"], CHUNK
    scale, share, dev = dk ** -0.5, H // c["Hk"], state["q"].device
    # the chunks: whose they are, their tokens, and which of these there are
    starts = torch.tensor(state["edges"], device=dev)
    n = int(state["edges"][-1])
    counts = (starts[1:] - starts[:-1] + C - 1) // C
    most = max((q - p + C - 1) // C for p, q in zip(state["edges"], state["edges"][1:]))
    base = torch.cumsum(counts, 0) - counts
    seq = torch.repeat_interleave(torch.arange(len(counts), device=dev), counts)
    at = starts[seq, None] + (torch.arange(len(seq), device=dev) - base[seq])[:, None] * C + torch.arange(C, device=dev)
    there = at < starts[seq + 1, None]
    at = torch.where(there, at, torch.zeros_like(at))
    rows = [(seqs, base[seqs] + i) for i in range(most) for seqs in [(counts > i).nonzero()[:, 0]]]

    def chunked(x):  # [n, H, d] -> [chunks, H, C, d]
        return (x[at] * there[..., None, None]).transpose(1, 2).contiguous()

    def back(x, like):  # the reverse, summed over the heads that shared it
        x = x.transpose(1, 2)[there]
        out = torch.empty_like(x)
        out[at[there]] = x
        if like.shape[1] != H:
            out = out.view(n, like.shape[1], share, -1).sum(2)
        return out.to(like.dtype)

    q, k = (chunked(state[x].float().repeat_interleave(share, 1)) for x in "qk")
    v = chunked(state["v"].float())
    log_a, slope, eta, eta_slope = (chunked(x[..., None]) for x in _gate_and_rate(state))
    G = torch.cumsum(log_a[..., 0], -1)
    R = torch.exp((G[..., None] - G[..., None, :]).tril()).tril()
    g, rest, last = torch.exp(G)[..., None], torch.exp(G[..., -1:] - G)[..., None], torch.exp(G[..., -1])[..., None, None]
    below = R.tril(-1) * (k @ k.transpose(2, 3).contiguous())
    A = eta * below
    inverse = torch.zeros_like(A)  # of 1 + A, row by row
    inverse[..., 0, 0] = 1
    for i in range(1, C):
        inverse[..., i, :i] = -(A[..., i, None, :i] @ inverse[..., :i, :i])[..., 0, :]
        inverse[..., i, i] = 1
    W, u = inverse @ (eta * g * k), inverse @ (eta * v)
    kT = (rest * k).transpose(2, 3).contiguous()
    qg = scale * g * q
    S = state["s0"].clone()
    train = c["op"] == "delta_train"
    before = torch.empty((len(seq), H, dk, dv), device=dev) if train else None
    o = scale * (R * (q @ k.transpose(2, 3).contiguous()))  # the scores, for now
    P, o = o, torch.empty_like(v)
    for seqs, ids in rows:
        Si = S[seqs]
        if train:
            before[ids] = Si
        ui = u[ids] - W[ids] @ Si
        u[ids] = ui
        o[ids] = qg[ids] @ Si + P[ids] @ ui
        S[seqs] = last[ids] * Si + kT[ids] @ ui
    out = {"o": back(o, state["v"]), "s_final": S}
    if not train:
        return out
    # dS runs from the end; du is the gradient of u, y that of the right-hand side over eta
    d_o = chunked(state["d_o"].float())
    dS = state["d_sfinal"].clone()
    after = torch.empty_like(before)
    du = P.transpose(2, 3).contiguous() @ d_o
    Wt, qt, kr = W.transpose(2, 3).contiguous(), qg.transpose(2, 3).contiguous(), rest * k
    for seqs, ids in reversed(rows):
        Si = dS[seqs]
        after[ids] = Si
        d = du[ids] + kr[ids] @ Si
        du[ids] = d
        dS[seqs] = last[ids] * Si + qt[ids] @ d_o[ids] - Wt[ids] @ d
    y = inverse.transpose(2, 3).contiguous() @ du
    ut = u.transpose(2, 3).contiguous()
    dP = scale * R * (d_o @ ut)
    dA = -(y @ ut).tril(-1)
    M = dA * eta * R
    E, F = dP * (q @ k.transpose(2, 3).contiguous()), M * (k @ k.transpose(2, 3).contiguous())
    bT, aT = before.transpose(2, 3).contiguous(), after.transpose(2, 3).contiguous()
    dq_in = scale * g * (d_o @ bT)
    dk_in, dk_out = -g * eta * (y @ bT), rest * (u @ aT)
    dq = dq_in + dP @ k
    dk_ = dk_in + dk_out + dP.transpose(2, 3).contiguous() @ q + (M + M.transpose(2, 3)).contiguous() @ k
    H_ = (dk_out * k).sum(-1)
    dG = (dq_in * q).sum(-1) + (dk_in * k).sum(-1) - H_ + E.sum(-1) - E.sum(-2) + F.sum(-1) - F.sum(-2)
    end = last[..., 0, 0] * (before * after).sum((-1, -2)) + H_.sum(-1)
    d_log = torch.flip(torch.cumsum(torch.flip(dG, [-1]), -1), [-1]) + end[..., None]
    error = v - g * (k @ before) - below @ u  # v - S'^T k
    out.update(dq=back(dq, state["q"]), dk=back(dk_, state["k"]), dv=back(eta * y, state["v"]),
               dgate=back(d_log[..., None] * slope, state["gate"][..., None])[..., 0],
               dbeta=back((y * error).sum(-1, keepdim=True) * eta * eta_slope, state["beta"][..., None])[..., 0], ds0=dS)
    return out


def _rotate(x, cos, sin, pairing):
    """The pairs of the first columns of x [n, H, d] turned by their angles; the others as they are."""
    half = cos.shape[-1]
    a, b = (x[..., :half], x[..., half:2 * half]) if pairing == "half" else (x[..., 0:2 * half:2], x[..., 1:2 * half:2])
    u, v = a * cos - b * sin, a * sin + b * cos
    turned = torch.cat([u, v], -1) if pairing == "half" else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _plain_qk(state):
    c = state["case"]
    d = c["d"]
    angle = state["pos"].double()[:, None] * state["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    out = {}
    for name in "qk":
        x, w = state[name].float(), state["w" + name]
        if c["norm"] == "none":
            rstd = torch.ones_like(x[..., :1])
        else:
            total = (x * x).sum(-1, keepdim=True)
            rstd = 1 / torch.sqrt((total / d if c["norm"] == "rms" else total) + EPS)
        hat = x * rstd
        y = hat if w is None else hat * w
        out["y" + name] = _rotate(y, cos, sin, c["pairing"]).to(state[name].dtype)
        if c["op"] == "qk_train":
            dy = _rotate(state["dy" + name].float(), cos, -sin, c["pairing"])
            dhat = dy if w is None else dy * w
            if c["norm"] == "none":
                dx = dhat
            else:
                dx = rstd * (dhat - hat * (dhat * hat).sum(-1, keepdim=True) / (d if c["norm"] == "rms" else 1))
            out["d" + name] = dx.to(state[name].dtype)
            if w is not None:
                out["dw" + name] = (dy * hat).sum((0, 1))
    return out


def work(case):
    """Each call's inputs read once and its outputs written once (a training step is a forward call and, later, a backward call)."""
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("qk"):
        n = case["tokens"] * (case["Hq"] + case["Hk"]) * case["d"]
        small = case["tokens"] * 4 + case["rot"] * 2 + (8 * case["d"] if case["weight"] else 0)
        if case["op"] == "qk_fwd":
            return {"bytes": 2 * e * n + small, "flops": 8 * n}
        return {"bytes": 5 * e * n + 2 * small + (8 * case["d"] if case["weight"] else 0), "flops": 24 * n}
    H, Hk, dk, dv = case["H"], case["Hk"], case["dk"], case["dv"]
    B = case["rows"] if "rows" in case else case["B"]
    n = B if "rows" in case else case["T"] if case["packed"] else B * case["T"]
    io = e * n * (2 * Hk * dk + H * dv + 2 * H)  # q, k, v, gate, beta
    o, state = e * n * H * dv, 4 * B * H * dk * dv
    # per token and head: the decay, the error, the update and the query, on dk x dv values
    flops = 7 * n * H * dk * dv
    if case["op"] != "delta_train":
        return {"bytes": io + o + 2 * state + (4 * B if "rows" in case else 0), "flops": flops}
    return {"bytes": 3 * io + 2 * o + 4 * state, "flops": 3 * flops}


def exact(case, seed):
    """The definitions, token by token, in 64 bits."""
    s = prepare(case, seed)
    if case["op"].startswith("qk"):
        return _exact_qk(s)
    if case["op"] == "delta_step":
        at = s["slots"].long()
        pool = s["s"].double()
        o, pool[at] = _token(_coefficients64(s), slice(None), pool[at])[:2]
        return {"o": o, "s": pool}
    # a token's steps take about 10 kernels forward, 25 more with the gradients
    loops = case["T"] if not case["packed"] else sum(q - p for p, q in zip(s["edges"], s["edges"][1:]))
    return _exact_delta(s) if loops * (4 if case["op"] == "delta_train" else 1) <= 140_000 else None


def _coefficients64(s):
    c = s["case"]
    z, b = s["gate"].double(), s["beta"].double()
    share = c["H"] // c["Hk"]
    a = torch.sigmoid(z) if c["gate"] == "sigmoid" else z.exp()
    return dict(q=s["q"].double().repeat_interleave(share, 1) * c["dk"] ** -0.5, k=s["k"].double().repeat_interleave(share, 1), v=s["v"].double(),
                a=a, eta=torch.sigmoid(b), da=a * torch.sigmoid(-z) if c["gate"] == "sigmoid" else a, deta=torch.sigmoid(b) * torch.sigmoid(-b))


def _token(x, at, S):
    """o, the state after the token(s) `at`, the decayed state before them and the error."""
    old = x["a"][at][..., None, None] * S
    e = x["v"][at] - (old * x["k"][at][..., None]).sum(-2)
    S = torch.addcmul(old, x["k"][at][..., None], (x["eta"][at][..., None] * e)[..., None, :])
    return (S * x["q"][at][..., None]).sum(-2), S, old, e


def _exact_delta(s):
    c = s["case"]
    x = _coefficients64(s)
    n, H, dk, dv = x["v"].shape[0], c["H"], c["dk"], c["dv"]
    train = c["op"] == "delta_train"
    f64 = dict(dtype=torch.float64, device=DEVICE)
    out = {"o": torch.empty((n, H, dv), **f64), "s_final": s["s0"].double()}
    if train:
        d_o = s["d_o"].double()
        out.update(dq=torch.empty((n, H, dk), **f64), dk=torch.empty((n, H, dk), **f64), dv=torch.empty((n, H, dv), **f64),
                   dgate=torch.empty((n, H), **f64), dbeta=torch.empty((n, H), **f64), ds0=s["d_sfinal"].double())
    # dense sequences walk side by side, packed ones one after the other
    if c["packed"]:
        walks = [(i, [slice(t, t + 1) for t in range(p, q)]) for i, (p, q) in enumerate(zip(s["edges"], s["edges"][1:]))]
        walks = [(slice(i, i + 1), ts) for i, ts in walks]
    else:
        walks = [(slice(None), [slice(t, None, c["T"]) for t in range(c["T"])])]
    for i, ts in walks:
        S, kept = out["s_final"][i].clone(), []
        for j, at in enumerate(ts):
            if train and j % 64 == 0:
                kept.append(S)
            out["o"][at], S = _token(x, at, S)[:2]
        out["s_final"][i] = S
        if not train:
            continue
        dS = out["ds0"][i]
        for j0 in range((len(ts) - 1) // 64 * 64, -1, -64):
            S, run_ = kept[j0 // 64], []
            for at in ts[j0:j0 + 64]:
                _, after, old, e = _token(x, at, S)
                run_.append((S, after, old, e))
                S = after
            for at, (first, after, old, e) in reversed(list(zip(ts[j0:j0 + 64], run_))):
                k, g = x["k"][at][..., None], d_o[at][..., None, :]
                dS = dS + x["q"][at][..., None] * g
                out["dq"][at] = (after * g).sum(-1)
                toward = (dS * k).sum(-2)  # dS^T k
                eta = x["eta"][at][..., None]
                out["dbeta"][at] = (toward * e).sum(-1) * x["deta"][at]
                de = eta * toward
                out["dv"][at] = de
                out["dk"][at] = (dS * (eta * e)[..., None, :]).sum(-1) - (old * de[..., None, :]).sum(-1)
                dS = dS - k * de[..., None, :]
                out["dgate"][at] = (dS * first).sum((-1, -2)) * x["da"][at]
                dS = x["a"][at][..., None, None] * dS
        out["ds0"][i] = dS
    if train:
        out["dq"] = (out["dq"] * dk ** -0.5).view(n, c["Hk"], -1, dk).sum(2)
        out["dk"] = out["dk"].view(n, c["Hk"], -1, dk).sum(2)
    return out


def _exact_qk(s):
    c = s["case"]
    half, d = c["rot"] // 2, c["d"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEVICE), s["pos"].double()[:, None] * s["inv_freq"].double())[:, None]

    def rotate(x, by):
        """The pairs as complex numbers, times e^{i angle}."""
        head = x[..., :2 * half]
        pairs = head.unflatten(-1, (2, half)).transpose(-1, -2) if c["pairing"] == "half" else head.unflatten(-1, (half, 2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * by)
        z = z.transpose(-1, -2) if c["pairing"] == "half" else z
        return torch.cat([z.flatten(-2), x[..., 2 * half:]], -1)

    out = {}
    for name in "qk":
        x = s[name].double().requires_grad_(c["op"] == "qk_train")
        w = s["w" + name]
        w = None if w is None else w.double().requires_grad_(c["op"] == "qk_train")
        size = dict(none=lambda: 1.0, rms=lambda: ((x ** 2).mean(-1, keepdim=True) + EPS) ** -0.5,
                    l2=lambda: ((x ** 2).sum(-1, keepdim=True) + EPS) ** -0.5)[c["norm"]]()
        y = x * size * (1.0 if w is None else w)
        y = rotate(y, turn) if half else y
        out["y" + name] = y.detach()
        if c["op"] == "qk_train":
            grads = torch.autograd.grad(y, [x] if w is None else [x, w], s["dy" + name].double())
            out["d" + name] = grads[0]
            if w is not None:
                out["dw" + name] = grads[1]
    return out
