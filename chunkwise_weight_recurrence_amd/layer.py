"""Device plumbing around the C ABI: move seeded inputs to HBM, allocate
outputs and workspace with torch, and call libttt.  No arithmetic of the layer
happens here -- torch only provides device memory and the stream.
"""
from __future__ import annotations

import math

import numpy as np

from . import binding as B


def _torch():
    import torch
    return torch


def to_device(arr, device="cuda"):
    """numpy payload -> torch tensor on the device (uint16 arrays are bf16 bit patterns)."""
    torch = _torch()
    if arr is None:
        return None
    if arr.dtype == np.uint16:
        t = torch.from_numpy(np.ascontiguousarray(arr).view(np.int16)).view(torch.bfloat16)
    else:
        t = torch.from_numpy(np.ascontiguousarray(arr))
    return t.to(device)


def to_f64(t):
    """torch tensor (bf16 or f32) -> numpy float64."""
    torch = _torch()
    return t.detach().to(torch.float32).cpu().numpy().astype(np.float64)


def desc_from_cfg(cfg):
    return B.make_desc(cfg["B"], cfg["H"], cfg["T"], cfg["dk"], cfg["dv"], cfg["C"],
                       dtype=cfg["dtype"], loss=cfg["loss"], act=cfg["act"], decay=cfg["decay"],
                       lr_bias=cfg["b"])


class TTTLayerBuffers:
    """Device copies of one input set plus every output and workspace buffer.

    With ``saved=True`` (the default) the forward keeps the library's saved
    context for the backward when the problem has one; ``saved=False`` makes
    the backward recompute the forward's chunk intermediates.
    """

    def __init__(self, inp, device="cuda", with_bwd=None, saved=True):
        torch = _torch()
        cfg = inp["cfg"]
        self.cfg = cfg
        self.desc = desc_from_cfg(cfg)
        Bn, H, T, dk, dv, C = cfg["B"], cfg["H"], cfg["T"], cfg["dk"], cfg["dv"], cfg["C"]
        self.nc = math.ceil(T / C) if T > 0 else 0
        io_dt = torch.bfloat16 if cfg["dtype"] == "bf16" else torch.float32
        f32 = torch.float32
        d = device
        self.q = to_device(inp["q_dev"], d)
        self.k = to_device(inp["k_dev"], d)
        self.v = to_device(inp["v_dev"], d)
        self.beta = to_device(inp["beta_dev"], d)
        self.gamma = to_device(inp.get("gamma_dev"), d)
        self.log_a = to_device(inp.get("log_a_dev"), d)
        self.w0 = to_device(inp.get("w0_dev"), d)
        self.o = torch.empty((Bn, H, T, dv), dtype=io_dt, device=d)
        self.w_final = torch.empty((Bn, H, dk, dv), dtype=f32, device=d)
        self.w_ckpt = torch.empty((Bn, H, self.nc, dk, dv), dtype=f32, device=d)
        ws_f = B.ttt_workspace_size(self.desc, B.ENTRY_FWD)
        self.ws_fwd = torch.empty(max(ws_f, 1), dtype=torch.uint8, device=d)
        self.has_bwd = cfg.get("bwd", False) if with_bwd is None else with_bwd
        if self.has_bwd:
            self.d_o = to_device(inp["d_o_dev"], d)
            self.dq = torch.empty((Bn, H, T, dk), dtype=io_dt, device=d)
            self.dk = torch.empty((Bn, H, T, dk), dtype=io_dt, device=d)
            self.dv = torch.empty((Bn, H, T, dv), dtype=io_dt, device=d)
            self.dbeta = torch.empty((Bn, H, T), dtype=f32, device=d)
            self.dgamma = torch.empty((Bn, H), dtype=f32, device=d) if cfg["decay"] == "scalar" else None
            self.dlog_a = torch.empty((Bn, H, T, dk), dtype=f32, device=d) \
                if cfg["decay"] == "vector" else None
            self.dw0 = torch.empty((Bn, H, dk, dv), dtype=f32, device=d)
            ws_b = B.ttt_workspace_size(self.desc, B.ENTRY_BWD)
            self.ws_bwd = torch.empty(max(ws_b, 1), dtype=torch.uint8, device=d)
        n_saved = B.ttt_saved_size(self.desc) if (saved and self.has_bwd) else 0
        self.saved = torch.empty(n_saved, dtype=torch.uint8, device=d) if n_saved else None

    def forward(self, stream=None):
        B.ttt_chunk_fwd(self.desc, self.q, self.k, self.v, self.beta, self.gamma, self.log_a, self.w0,
                        self.o, self.w_final, self.w_ckpt, self.saved, self.ws_fwd, stream=stream)

    def backward(self, stream=None, d_wfinal=None):
        B.ttt_chunk_bwd(self.desc, self.q, self.k, self.v, self.beta, self.gamma, self.log_a, self.w0,
                        self.w_ckpt, self.saved, self.d_o, d_wfinal, self.dq, self.dk, self.dv, self.dbeta,
                        self.dgamma, self.dlog_a, self.dw0, self.ws_bwd, stream=stream)


class MlpBuffers:
    """Device copies of one two-layer (TTT-MLP) input set, its outputs and workspace."""

    def __init__(self, inp, device="cuda", with_bwd=False, saved=True):
        torch = _torch()
        cfg = inp["cfg"]
        self.cfg = cfg
        self.desc = B.make_mlp_desc(cfg["B"], cfg["H"], cfg["T"], cfg["dk"], cfg["dh"], cfg["dv"], cfg["C"],
                                    dtype=cfg["dtype"], loss=cfg["loss"], act=cfg["act"], decay=cfg["decay"],
                                    lr_bias=cfg["b"])
        Bn, H, T, dk, dh, dv = cfg["B"], cfg["H"], cfg["T"], cfg["dk"], cfg["dh"], cfg["dv"]
        io_dt = torch.bfloat16 if cfg["dtype"] == "bf16" else torch.float32
        d = device
        self.q = to_device(inp["q_dev"], d)
        self.k = to_device(inp["k_dev"], d)
        self.v = to_device(inp["v_dev"], d)
        self.beta = to_device(inp["beta_dev"], d)
        self.gamma = to_device(inp.get("gamma_dev"), d)
        self.w1_0 = to_device(inp.get("w1_0_dev"), d)
        self.w2_0 = to_device(inp.get("w2_0_dev"), d)
        self.o = torch.empty((Bn, H, T, dv), dtype=io_dt, device=d)
        self.w1 = torch.empty((Bn, H, dk, dh), dtype=torch.float32, device=d)
        self.w2 = torch.empty((Bn, H, dh, dv), dtype=torch.float32, device=d)
        self.ws_bytes = B.ttt_mlp_workspace_size(self.desc)
        self.ws = torch.empty(max(self.ws_bytes, 1), dtype=torch.uint8, device=d)
        self.has_bwd = with_bwd
        self.w1_ckpt = self.w2_ckpt = None
        if with_bwd:
            nc = -(-T // cfg["C"]) if T > 0 else 0
            f32 = torch.float32
            self.w1_ckpt = torch.empty((Bn, H, nc, dk, dh), dtype=f32, device=d)
            self.w2_ckpt = torch.empty((Bn, H, nc, dh, dv), dtype=f32, device=d)
            self.dq = torch.empty((Bn, H, T, dk), dtype=io_dt, device=d)
            self.dk = torch.empty((Bn, H, T, dk), dtype=io_dt, device=d)
            self.dv = torch.empty((Bn, H, T, dv), dtype=io_dt, device=d)
            self.dbeta = torch.empty((Bn, H, T), dtype=f32, device=d)
            self.dgamma = torch.empty((Bn, H), dtype=f32, device=d) if cfg["decay"] == "scalar" else None
            self.dw1 = torch.empty((Bn, H, dk, dh), dtype=f32, device=d)
            self.dw2 = torch.empty((Bn, H, dh, dv), dtype=f32, device=d)
            self.ws_bwd_bytes = B.ttt_mlp_bwd_workspace_size(self.desc)
            self.ws_bwd = torch.empty(max(self.ws_bwd_bytes, 1), dtype=torch.uint8, device=d)
        n_saved = B.ttt_mlp_saved_size(self.desc) if (with_bwd and saved) else 0
        self.saved = torch.empty(n_saved, dtype=torch.uint8, device=d) if n_saved else None

    def forward(self, stream=None):
        B.ttt_mlp_chunk_fwd(self.desc, self.q, self.k, self.v, self.beta, self.gamma, self.w1_0, self.w2_0,
                            self.o, self.w1, self.w2, self.w1_ckpt, self.w2_ckpt, self.saved, self.ws,
                            self.ws_bytes, stream=stream)

    def backward(self, d_o, d_w1final=None, d_w2final=None, stream=None):
        """The outer backward from the forward's checkpoints; fills dq, dk, dv, dbeta,
        dgamma (scalar decay), dw1 and dw2."""
        B.ttt_mlp_chunk_bwd(self.desc, self.q, self.k, self.v, self.beta, self.gamma, self.w1_ckpt, self.w2_ckpt,
                            self.saved, d_o, d_w1final, d_w2final, self.dq, self.dk, self.dv, self.dbeta, self.dgamma, self.dw1,
                            self.dw2, self.ws_bwd, self.ws_bwd_bytes, stream=stream)


class InplaceBuffers:
    """Device copies of In-Place inputs; w_down is reset from w0 by reset().

    With ``clip_tau`` or ``doc_lens`` in the config (or ``guarded=True``) the
    guarded entry point runs, and w0 is also the state documents restart from.
    """

    def __init__(self, inp, device="cuda", workspace=True, guarded=None):
        from .workloads import inplace_doc_starts
        torch = _torch()
        cfg = inp["cfg"]
        self.cfg = cfg
        self.guarded = bool(cfg.get("clip_tau") or cfg.get("doc_lens")) if guarded is None else guarded
        self.doc_starts = inplace_doc_starts(cfg)[1]
        self.z = to_device(inp["z_dev"], device)
        self.vhat = to_device(inp["vhat_dev"], device)
        self.w0 = to_device(inp["w0_dev"], device)
        self.w = self.w0.clone()
        Bn, T, dm = cfg["B"], cfg["T"], cfg["d_model"]
        self.o = torch.empty((Bn, T, dm), dtype=torch.bfloat16, device=device)
        size = B.inplace_ttt_guarded_workspace_size if self.guarded else B.inplace_ttt_workspace_size
        n_ws = size(Bn, T, dm, cfg["d_ff"], cfg["C"]) if workspace else 0
        self.ws = torch.empty(n_ws, dtype=torch.uint8, device=device) if n_ws else None
        self.ws_bytes = n_ws

    def reset(self):
        self.w.copy_(self.w0)

    def backward(self, d_o, d_wfinal=None, stream=None):
        """The backward from the state the last forward left in ``self.w``
        (inplace_ttt_bwd, or inplace_ttt_bwd_guarded for the guarded forward);
        returns (dz, dvhat, dw0) device tensors.  Guarded, ``self.dw_init``
        then holds dL/dw_init over the documents after each sequence's first
        (w0 is also the state they restart from, so its total derivative is
        dw0 + dw_init)."""
        torch = _torch()
        c = self.cfg
        dev = self.w.device
        Bn, T, dm, dff = c["B"], c["T"], c["d_model"], c["d_ff"]
        if not hasattr(self, "dz"):
            self.dz = torch.empty((Bn, T, dff), dtype=torch.bfloat16, device=dev)
            self.dvhat = torch.empty((Bn, T, dm), dtype=torch.bfloat16, device=dev)
            self.dw0 = torch.empty((Bn, dm, dff), dtype=torch.float32, device=dev)
            size = B.inplace_ttt_bwd_guarded_workspace_size if self.guarded else B.inplace_ttt_bwd_workspace_size
            n = size(Bn, T, dm, dff, c["C"])
            self.ws_bwd = torch.empty(max(n, 1), dtype=torch.uint8, device=dev)
            self.ws_bwd_bytes = n
            self.dw_init = torch.empty((Bn, dm, dff), dtype=torch.float32, device=dev) if self.guarded else None
        if self.guarded:
            B.inplace_ttt_bwd_guarded(Bn, T, dm, dff, c["C"], c["eta"], c.get("clip_tau") or 0.0, self.doc_starts,
                                      self.z, self.vhat, self.w0, self.w0, self.w, d_o, d_wfinal, self.dz,
                                      self.dvhat, self.dw0, self.dw_init, self.ws_bwd, self.ws_bwd_bytes,
                                      stream=stream)
        else:
            B.inplace_ttt_bwd(Bn, T, dm, dff, c["C"], c["eta"], self.z, self.vhat, self.w, d_o, d_wfinal, self.dz,
                              self.dvhat, self.dw0, self.ws_bwd, self.ws_bwd_bytes, stream=stream)
        return self.dz, self.dvhat, self.dw0

    def forward(self, stream=None):
        c = self.cfg
        if self.guarded:
            B.inplace_ttt_fwd_guarded(c["B"], c["T"], c["d_model"], c["d_ff"], c["C"], c["eta"],
                                      c.get("clip_tau") or 0.0, self.doc_starts, self.z, self.vhat, self.w0,
                                      self.w, self.o, self.ws, self.ws_bytes, stream=stream)
        else:
            B.inplace_ttt_fwd(c["B"], c["T"], c["d_model"], c["d_ff"], c["C"], c["eta"], self.z, self.vhat,
                              self.w, self.o, self.ws, self.ws_bytes, stream=stream)


def _row_distance(x):
    """Elements from one row of ``x`` ([..., D]) to the next: the stride of its innermost leading axis of more than one."""
    if x.numel() > 0:
        for i in range(x.dim() - 2, -1, -1):
            if x.shape[i] > 1:
                return x.stride(i)
    return x.shape[-1]


class RecurrenceBuffers:
    """Outputs and workspace of the gated linear recurrence over x and gate ([B,T,D], or packed [T,D]).

    ``x`` and ``gate`` are device tensors whose rows may be strided (two halves
    of one projection).  ``seq_starts``: int32 device tensor of B + 1 row
    positions for packed sequences.  ``h0``: [B,D] float32 or None."""

    def __init__(self, x, gate, kind="sigmoid", input="convex", h0=None, seq_starts=None, with_bwd=False):
        torch = _torch()
        packed = seq_starts is not None
        if x.dim() < (2 if packed else 3) or math.prod(x.shape[:1 if packed else 2]) * x.shape[-1] != x.numel():
            raise ValueError(f"x must be {'[T,D]' if packed else '[B,T,D]'} (got shape {tuple(x.shape)})")
        if gate.shape[-1:] != x.shape[-1:] or gate.numel() != x.numel():
            raise ValueError(f"gate must have x's shape {tuple(x.shape)} (got {tuple(gate.shape)})")
        D = x.shape[-1]
        Bn, T = (seq_starts.numel() - 1, x.shape[0]) if packed else x.shape[:2]
        self.x, self.gate, self.h0, self.seq_starts = x, gate, h0, seq_starts
        self.desc = B.make_rec_desc(Bn, T, D, dtype="bf16" if x.dtype == torch.bfloat16 else "f32", gate=kind,
                                    input=input, packed=packed, ldx=_row_distance(x), ldg=_row_distance(gate))
        d = x.device
        self.o = torch.empty(x.shape, dtype=x.dtype, device=d)
        self.h_final = torch.empty((Bn, D), dtype=torch.float32, device=d)
        size = B.ttt_recurrence_workspace_size(self.desc, B.ENTRY_FWD)
        self.saved = None
        if with_bwd:
            size = max(size, B.ttt_recurrence_workspace_size(self.desc, B.ENTRY_BWD))
            self.saved = torch.empty(B.ttt_recurrence_saved_size(self.desc), dtype=torch.uint8, device=d)
            self.dx = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=d)
            self.dgate = torch.empty_strided(gate.shape, gate.stride(), dtype=gate.dtype, device=d)
            self.dh0 = torch.empty((Bn, D), dtype=torch.float32, device=d)
        self.ws = torch.empty(max(size, 1), dtype=torch.uint8, device=d)

    def forward(self, stream=None):
        B.ttt_recurrence_fwd(self.desc, self.x, self.gate, self.h0, self.seq_starts, self.o, self.h_final, self.saved,
                             self.ws, stream=stream)

    def backward(self, d_o, d_hfinal=None, stream=None):
        """Fills dx, dgate (with the strides of x and gate) and dh0."""
        B.ttt_recurrence_bwd(self.desc, self.x, self.gate, self.h0, self.seq_starts, self.saved, d_o, d_hfinal, self.dx,
                             self.dgate, self.dh0, self.ws, stream=stream)


class LayerNormBuffers:
    """Outputs and workspace of the layer norm over the rows of ``x`` ([..., D], rows may be strided).

    ``w``, ``b``: [groups, D] float32 or None; row i has group (i / period) %
    groups.  ``res``: the residual stream or None; ``self.r`` is then the new one."""

    def __init__(self, x, w=None, b=None, res=None, groups=1, period=1, eps=1e-5, with_bwd=False):
        torch = _torch()
        if res is not None and (res.shape[-1:] != x.shape[-1:] or res.numel() != x.numel()):
            raise ValueError(f"res must have x's shape {tuple(x.shape)} (got {tuple(res.shape)})")
        D = x.shape[-1]
        rows = x.numel() // D
        f32, d = torch.float32, x.device
        self.x, self.w, self.b, self.res = x, w, b, res
        dtype = "bf16" if x.dtype == torch.bfloat16 else "f32"
        self.desc = B.make_ln_desc(rows, D, dtype=dtype, groups=groups, period=period, eps=eps, ldx=_row_distance(x))
        # the backward reads the rows that were normalised: the dense r where there is a residual
        self.desc_bwd = self.desc if res is None else B.make_ln_desc(rows, D, dtype=dtype, groups=groups, period=period,
                                                                     eps=eps)
        self.y = torch.empty(x.shape, dtype=x.dtype, device=d)
        self.r = torch.empty(x.shape, dtype=x.dtype, device=d) if res is not None else None
        self.mean = self.rstd = None
        if with_bwd:
            self.mean = torch.empty(rows, dtype=f32, device=d)
            self.rstd = torch.empty(rows, dtype=f32, device=d)
            self.dx = torch.empty_like(self.r) if res is not None else \
                torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=d)
            self.dw = torch.empty((groups, D), dtype=f32, device=d)
            self.db = torch.empty((groups, D), dtype=f32, device=d)
            self.ws = torch.empty(B.ttt_layernorm_workspace_size(self.desc_bwd), dtype=torch.uint8, device=d)

    def forward(self, stream=None):
        B.ttt_layernorm_fwd(self.desc, self.x, self.res, self.w, self.b, self.y, self.r, self.mean, self.rstd,
                            stream=stream)

    def backward(self, dy, dr=None, stream=None):
        """Fills dx (also the residual's gradient), dw and db."""
        B.ttt_layernorm_bwd(self.desc_bwd, self.x if self.r is None else self.r, self.w, self.mean, self.rstd, dy, dr,
                            self.dx, self.dw, self.db, self.ws, stream=stream)


def _token_distance(x):
    """Elements from one token of ``x`` ([..., H, d], the heads of a token side by side) to the next."""
    H, d = x.shape[-2:]
    if (H > 1 and x.stride(-2) != d) or (d > 1 and x.stride(-1) != 1):
        raise ValueError(f"the heads of a token must lie side by side (got shape {tuple(x.shape)}, strides {x.stride()})")
    if x.numel() > 0:
        for i in range(x.dim() - 3, -1, -1):
            if x.shape[i] > 1:
                return x.stride(i)
    return H * d


def _check_heads(name, x, like):
    """A tensor ``x`` has the tokens, heads and channels of ``like``, the tokens' axes as they may be."""
    if hasattr(x, "shape") and (x.shape[-2:] != like.shape[-2:] or x.numel() != like.numel()):
        raise ValueError(f"{name} must have the heads and channels of {tuple(like.shape)} (got {tuple(x.shape)})")


class DeltaBuffers:
    """Outputs and workspace of the gated delta rule over q, k [B,T,Hk,dk] and v [B,T,H,dv], or packed [T,Hk,dk], [T,H,dv].

    Device tensors whose tokens may be strided (slices of one projection).
    ``gate`` ([..,H], or None for no decay) and ``beta`` ([..,H]).  ``seq_starts``:
    int32 device tensor of B + 1 positions for packed sequences.  ``s0``:
    [B,H,dk,dv] float32 or None."""

    def __init__(self, q, k, v, gate, beta, kind="sigmoid", s0=None, seq_starts=None, scale=None, lr_max=1.0, lr_bias=0.0,
                 with_bwd=False):
        torch = _torch()
        packed = seq_starts is not None
        lead = 1 if packed else 2
        if q.dim() != lead + 2 or k.shape != q.shape or v.dim() != lead + 2 or v.shape[:lead] != q.shape[:lead]:
            raise ValueError(f"q and k must be {'[T,Hk,dk]' if packed else '[B,T,Hk,dk]'} and v {'[T,H,dv]' if packed else '[B,T,H,dv]'} "
                             f"(got shapes {tuple(q.shape)}, {tuple(k.shape)}, {tuple(v.shape)})")
        for name, x in (("gate", gate), ("beta", beta)):
            if x is not None and x.shape != v.shape[:-1]:
                raise ValueError(f"{name} must have shape {tuple(v.shape[:-1])} (got {tuple(x.shape)})")
        Hk, dk = q.shape[-2:]
        H, dv = v.shape[-2:]
        Bn, T = (seq_starts.numel() - 1, q.shape[0]) if packed else q.shape[:2]
        f32, d = torch.float32, q.device
        self._state_shape = (Bn, H, dk, dv)
        self._check_state("s0", s0)
        self.q, self.k, self.v, self.gate, self.beta, self.s0, self.seq_starts = q, k, v, gate, beta, s0, seq_starts
        self.desc = B.make_delta_desc(Bn, T, H, dk, dv, Hk=Hk, dtype="bf16" if q.dtype == torch.bfloat16 else "f32", gate=kind,
                                      packed=packed, scale=scale, lr_max=lr_max, lr_bias=lr_bias, ldq=_token_distance(q),
                                      ldk=_token_distance(k), ldv=_token_distance(v),
                                      ldg=0 if gate is None else _row_distance(gate), ldb=_row_distance(beta))
        self.o = torch.empty(v.shape, dtype=v.dtype, device=d)
        self.s_final = torch.empty((Bn, H, dk, dv), dtype=f32, device=d)
        size = B.ttt_delta_workspace_size(self.desc, B.ENTRY_FWD)
        self.saved = None
        if with_bwd:
            size = max(size, B.ttt_delta_workspace_size(self.desc, B.ENTRY_BWD))
            self.saved = torch.empty(B.ttt_delta_saved_size(self.desc), dtype=torch.uint8, device=d)
            self.dq, self.dk, self.dv, self.dbeta = (torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=d)
                                                     for x in (q, k, v, beta))
            self.dgate = None if gate is None else torch.empty_strided(gate.shape, gate.stride(), dtype=gate.dtype, device=d)
            self.ds0 = torch.empty((Bn, H, dk, dv), dtype=f32, device=d)
        self.ws = torch.empty(max(size, 1), dtype=torch.uint8, device=d)

    def _check_state(self, name, x):
        if x is not None and x.shape != self._state_shape:
            raise ValueError(f"{name} must have shape {self._state_shape} (got {tuple(x.shape)})")

    def forward(self, stream=None):
        B.ttt_delta_fwd(self.desc, self.q, self.k, self.v, self.gate, self.beta, self.s0, self.seq_starts, self.o, self.s_final,
                        self.saved, self.ws, stream=stream)

    def backward(self, d_o, d_sfinal=None, stream=None):
        """Fills dq, dk, dv, dgate and dbeta (with the strides of q, k, v, gate and beta) and ds0."""
        _check_heads("d_o", d_o, self.v)
        self._check_state("d_sfinal", d_sfinal)
        B.ttt_delta_bwd(self.desc, self.q, self.k, self.v, self.gate, self.beta, self.seq_starts, self.saved, d_o, d_sfinal,
                        self.dq, self.dk, self.dv, self.dgate, self.dbeta, self.ds0, self.ws, stream=stream)


class QkNormBuffers:
    """Outputs and workspace of the norm and rotation of q [..,Hq,d] and k [..,Hk,d] (tokens may be strided).

    ``wq``, ``wk``: [d] float32 or None; ``positions``: int32 [tokens] or None (then token t is at t % period);
    ``inv_freq``: float32 [rot / 2] or None for no rotation."""

    def __init__(self, q, k, wq=None, wk=None, positions=None, inv_freq=None, norm="rms", pairing="half", period=0, eps=1e-6,
                 rot_scale=1.0, with_bwd=False):
        torch = _torch()
        if q.dim() < 3 or k.shape[:-2] != q.shape[:-2] or k.shape[-1] != q.shape[-1]:
            raise ValueError(f"q and k must be [..,Hq,d] and [..,Hk,d] (got shapes {tuple(q.shape)}, {tuple(k.shape)})")
        for name, w in (("wq", wq), ("wk", wk)):
            if w is not None and w.shape != q.shape[-1:]:
                raise ValueError(f"{name} must have shape {tuple(q.shape[-1:])} (got {tuple(w.shape)})")
        if positions is not None and positions.numel() != math.prod(q.shape[:-2]):
            raise ValueError(f"positions must be one a token (got shape {tuple(positions.shape)} for {math.prod(q.shape[:-2])})")
        f32, d = torch.float32, q.device
        self.q, self.k, self.wq, self.wk, self.positions, self.inv_freq = q, k, wq, wk, positions, inv_freq
        rot = 0 if inv_freq is None else 2 * inv_freq.numel()
        self.desc = B.make_qknorm_desc(math.prod(q.shape[:-2]), q.shape[-2], k.shape[-2], q.shape[-1], rot=rot, pairing=pairing,
                                       norm=norm, dtype="bf16" if q.dtype == torch.bfloat16 else "f32", period=period, eps=eps,
                                       rot_scale=rot_scale, ldq=_token_distance(q), ldk=_token_distance(k))
        self.yq, self.yk = (torch.empty(x.shape, dtype=x.dtype, device=d) for x in (q, k))
        if with_bwd:
            self.dq, self.dk = (torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=d) for x in (q, k))
            self.dwq, self.dwk = (None if w is None else torch.empty(q.shape[-1], dtype=f32, device=d) for w in (wq, wk))
            self.ws = torch.empty(B.ttt_qknorm_workspace_size(self.desc), dtype=torch.uint8, device=d)

    def forward(self, stream=None):
        B.ttt_qknorm_fwd(self.desc, self.q, self.k, self.wq, self.wk, self.positions, self.inv_freq, self.yq, self.yk,
                         stream=stream)

    def backward(self, dyq, dyk, stream=None):
        """Fills dq and dk (with the strides of q and k), dwq and dwk."""
        _check_heads("dyq", dyq, self.q)
        _check_heads("dyk", dyk, self.k)
        B.ttt_qknorm_bwd(self.desc, self.q, self.k, self.wq, self.wk, self.positions, self.inv_freq, dyq, dyk, self.dq, self.dk,
                         self.dwq, self.dwk, self.ws, stream=stream)
