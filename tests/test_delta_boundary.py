"""Refusals of the gated delta rule's and the query and key norm's entry points and buffers (CPU): bad
arguments are rejected on the host, before any HIP call, with the documented status."""
import ctypes

import pytest
import torch

import chunkwise_weight_recurrence_amd as ttt
from chunkwise_weight_recurrence_amd import binding as B
from chunkwise_weight_recurrence_amd.layer import DeltaBuffers, QkNormBuffers

FAKE = 0x1000   # never dereferenced: every case below fails validation first or has nothing to do


def _desc(**kw):
    base = dict(B=3, T=300, H=4, dk=64, dv=32, Hk=2)
    base.update(kw)
    return B.make_delta_desc(**base)


def _fwd(d, **kw):
    p = dict(q=FAKE, k=FAKE, v=FAKE, gate=FAKE, beta=FAKE, s0=None, seq_starts=None, o=FAKE, s_final=None, saved=None, ws=FAKE,
             ws_bytes=1 << 40)
    p.update(kw)
    return B.lib().ttt_delta_fwd(ctypes.byref(d) if d is not None else None, *p.values(), None)


def _bwd(d, **kw):
    p = dict(q=FAKE, k=FAKE, v=FAKE, gate=FAKE, beta=FAKE, seq_starts=None, saved=FAKE, d_o=FAKE, d_sfinal=None, dq=FAKE, dk=FAKE,
             dv=FAKE, dgate=FAKE, dbeta=FAKE, ds0=None, ws=FAKE, ws_bytes=1 << 40)
    p.update(kw)
    return B.lib().ttt_delta_bwd(ctypes.byref(d), *p.values(), None)


def _step(d, **kw):
    p = dict(q=FAKE, k=FAKE, v=FAKE, gate=FAKE, beta=FAKE, slots=None, n_states=3, s=FAKE, s_new=FAKE, o=FAKE)
    p.update(kw)
    return B.lib().ttt_delta_step(ctypes.byref(d), *p.values(), None)


def _qk(**kw):
    base = dict(tokens=10, Hq=4, Hk=2, d=64)
    base.update(kw)
    return B.make_qknorm_desc(**base)


def _qfwd(d, **kw):
    p = dict(q=FAKE, k=FAKE, wq=None, wk=None, positions=None, inv_freq=FAKE, yq=2 * FAKE, yk=2 * FAKE)
    p.update(kw)
    return B.lib().ttt_qknorm_fwd(ctypes.byref(d) if d is not None else None, *p.values(), None)


def _qbwd(d, **kw):
    p = dict(q=FAKE, k=FAKE, wq=None, wk=None, positions=None, inv_freq=FAKE, dyq=FAKE, dyk=FAKE, dq=FAKE, dk=FAKE, dwq=FAKE,
             dwk=FAKE, ws=FAKE, ws_bytes=1 << 30)
    p.update(kw)
    return B.lib().ttt_qknorm_bwd(ctypes.byref(d), *p.values(), None)


def test_structs_and_enums_match_the_header():
    import os
    import re
    assert ctypes.sizeof(B.TTTDeltaDesc) == 88 and ctypes.sizeof(B.TTTQkNormDesc) == 64
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ttt.h")).read()
    for cls, prefix in ((B.HeadNorm, "TTT_HEADNORM_"), (B.RopePairs, "TTT_ROPE_"), (B.Kernel, "TTT_KERNEL_")):
        for m in cls:
            assert int(re.search(rf"\b{prefix}{m.name}\s*=\s*(\d+)", src).group(1)) == int(m)
    assert int(re.search(r"TTT_KERNEL_COUNT\s*=\s*(\d+)", src).group(1)) == len(B.Kernel)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(B=-1), -1, "B, T"), (dict(T=-1), -1, "B, T"), (dict(H=0, Hk=1), -1, "divisor"), (dict(Hk=3), -1, "divisor"),
    (dict(Hk=0), -1, "divisor"), (dict(dk=0), -1, "dk, dv"), (dict(dv=0), -1, "dk, dv"), (dict(packed=2), -1, "packed"),
    (dict(dtype=7), -1, "dtype"), (dict(gate=2), -1, "gate"), (dict(scale=float("inf")), -1, "finite"),
    (dict(lr_max=float("nan")), -1, "finite"), (dict(lr_bias=float("inf")), -1, "finite"), (dict(dk=257), -2, "dk, dv"),
    (dict(dv=257), -2, "dk, dv"), (dict(ldq=127), -1, "ldq"), (dict(ldk=1), -1, "ldq"), (dict(ldv=-128), -1, "ldq"),
    (dict(ldg=3), -1, "ldq"), (dict(ldb=3), -1, "ldq"), (dict(ldv=1 << 24), -2, "too large"),
    (dict(B=1 << 16, T=1 << 15), -2, "too large"), (dict(T=(1 << 30), B=1), -2, "too large"),
    (dict(B=1 << 23, T=1), -2, "too large"), (dict(B=(1 << 31) - 1, T=0, packed=True), -2, "too large"),
    (dict(H=1 << 18, Hk=1, dv=64), -2, "too large"),
    # a launch has fewer than 2^32 threads, 512 of them for a chunk and head or a sequence's columns
    (dict(B=1, T=1 << 27, H=4), -2, "too large"), (dict(B=1 << 20, T=1, H=4, dv=1), -2, "too large"),
    (dict(B=1 << 19, T=1, H=4, dv=32), -2, "too large"), (dict(ldq=(1 << 22) + 1), -2, "too large"),
])
def test_delta_desc(kw, code, msg):
    d = _desc(**kw)
    n = ctypes.c_size_t(0)
    for st in (_fwd(d), _bwd(d), _step(d), B.lib().ttt_delta_workspace_size(ctypes.byref(d), 0, ctypes.byref(n)),
               B.lib().ttt_delta_saved_size(ctypes.byref(d), ctypes.byref(n))):
        assert st == code and msg in ttt.ttt_last_error()


def test_delta_pointers_and_workspace():
    d, p = _desc(), _desc(packed=True)
    assert _fwd(None) == -1 and "desc is NULL" in ttt.ttt_last_error()
    for name in ("q", "k", "v", "beta", "o"):
        assert _fwd(d, **{name: None}) == -1 and "required" in ttt.ttt_last_error()
    for name in ("q", "k", "v", "beta", "saved", "d_o", "dq", "dk", "dv", "dbeta"):
        assert _bwd(d, **{name: None}) == -1 and "required" in ttt.ttt_last_error()
    for kw in (dict(gate=None), dict(dgate=None)):
        assert _bwd(d, **kw) == -1 and "go together" in ttt.ttt_last_error()
    for f in (_fwd, _bwd):
        assert f(p) == -1 and "seq_starts" in ttt.ttt_last_error()
        assert f(d, seq_starts=FAKE) == -1 and "seq_starts" in ttt.ttt_last_error()
        for name in ("q", "k", "v", "gate", "beta"):
            assert f(d, **{name: FAKE + 1}) == -1 and f"{name} must be aligned to its elements" in ttt.ttt_last_error()
        assert f(_desc(dtype="f32"), q=FAKE + 2) == -1 and "elements" in ttt.ttt_last_error()
        assert f(p, seq_starts=FAKE + 4) == -1 and "seq_starts must be 16-byte" in ttt.ttt_last_error()
        assert f(d, ws=None) == -3 and f(d, ws_bytes=16) == -3
    assert _fwd(d, o=FAKE + 8) == -1 and _bwd(d, d_o=FAKE + 8) == -1
    size = 3 * 4 * 64 * 32 * 4
    assert _fwd(d, s0=FAKE, s_final=FAKE) == -1 and "overlap" in ttt.ttt_last_error()
    assert _fwd(d, s0=FAKE, s_final=FAKE + size - 16) == -1
    assert _bwd(d, d_sfinal=FAKE + 16, ds0=FAKE) == -1 and "overlap" in ttt.ttt_last_error()
    n = ctypes.c_size_t(0)
    assert B.lib().ttt_delta_workspace_size(ctypes.byref(d), 2, ctypes.byref(n)) == -1
    assert B.lib().ttt_delta_workspace_size(ctypes.byref(d), 0, None) == -1
    assert B.lib().ttt_delta_saved_size(ctypes.byref(d), None) == -1


def test_delta_sizes_cover_any_lengths():
    """Packed sequences have room for the most chunks that any lengths make."""
    for dtype, C in (("bf16", 64), ("f32", 32)):
        dense = ttt.ttt_delta_saved_size(_desc(B=10, T=1, dtype=dtype))
        assert ttt.ttt_delta_saved_size(_desc(B=10, T=10, packed=True, dtype=dtype)) == dense   # ten of one token
        one = ttt.ttt_delta_saved_size(_desc(B=1, T=1, dtype=dtype))
        assert ttt.ttt_delta_saved_size(_desc(B=1, T=C, dtype=dtype)) == one < ttt.ttt_delta_saved_size(_desc(B=1, T=C + 1, dtype=dtype))


def test_delta_empty_problems_need_no_device():
    none = dict(q=None, k=None, v=None, gate=None, beta=None, o=None, ws=None, ws_bytes=0)
    assert _fwd(_desc(B=0, T=0), **none) == 0 and _fwd(_desc(T=0), **none) == 0
    assert _fwd(_desc(B=0, T=0, packed=True), **none) == 0 and _fwd(_desc(B=0, T=9, packed=True), **none) == 0
    gone = dict(q=None, k=None, v=None, gate=None, beta=None, saved=None, d_o=None, dq=None, dk=None, dv=None, dgate=None, dbeta=None)
    assert _bwd(_desc(T=0), **gone) == 0
    assert _step(_desc(B=0, T=1), q=None, s=None) == 0
    for d in (_desc(T=0), _desc(B=0)):
        assert ttt.ttt_delta_workspace_size(d, 0) == 0 and ttt.ttt_delta_workspace_size(d, 1) == 0


def test_delta_step_refusals():
    d = _desc(T=1)
    assert _step(_desc(T=2)) == -1 and "T = 1" in ttt.ttt_last_error()
    assert _step(_desc(T=1, packed=True)) == -1
    assert _step(d, n_states=2) == -1 and "n_states" in ttt.ttt_last_error()   # three rows without slots
    assert _step(d, n_states=-1) == -1
    assert _step(_desc(B=(1 << 20) + 1, T=1, H=1, Hk=1, dv=8, dk=8), slots=FAKE) == -2 and "slots" in ttt.ttt_last_error()
    for name in ("q", "k", "v", "beta", "s", "s_new", "o"):
        assert _step(d, **{name: None}) == -1 and "required" in ttt.ttt_last_error()
    assert _step(d, s=FAKE, s_new=FAKE + 3 * 4 * 64 * 32 * 4 - 16) == -1 and "overlap" in ttt.ttt_last_error()
    assert _step(d, slots=FAKE + 4) == -1 and _step(d, k=FAKE + 1) == -1 and _step(d, o=FAKE + 2) == -1


@pytest.mark.parametrize("kw,code,msg", [
    (dict(tokens=-1), -1, "tokens"), (dict(Hq=0), -1, "Hq"), (dict(Hk=-1), -1, "Hk"), (dict(d=0, rot=0), -1, "d must"),
    (dict(rot=3), -1, "rot"), (dict(rot=66), -1, "rot"), (dict(rot=-2), -1, "rot"), (dict(pairing=2), -1, "pairing"),
    (dict(norm=3), -1, "norm"), (dict(norm=-1), -1, "norm"), (dict(period=-1), -1, "period"), (dict(dtype=2), -1, "dtype"),
    (dict(eps=-1.0), -1, "eps"), (dict(eps=float("nan")), -1, "eps"), (dict(rot_scale=float("inf")), -1, "rot_scale"),
    (dict(ldq=255), -1, "ldq"), (dict(ldk=1), -1, "ldq"), (dict(d=514), -2, "too large"), (dict(ldq=1 << 24), -2, "too large"),
    (dict(tokens=1 << 31), -2, "too large"), (dict(Hq=1 << 20), -2, "too large"),
])
def test_qknorm_desc(kw, code, msg):
    d = _qk(**kw)
    n = ctypes.c_size_t(0)
    for st in (_qfwd(d), _qbwd(d), B.lib().ttt_qknorm_workspace_size(ctypes.byref(d), ctypes.byref(n))):
        assert st == code and msg in ttt.ttt_last_error()


def test_qknorm_pointers():
    d = _qk()
    assert _qfwd(None) == -1
    for name in ("q", "k", "yq", "yk"):
        assert _qfwd(d, **{name: None}) == -1 and "required" in ttt.ttt_last_error()
    for name in ("q", "k", "dyq", "dyk", "dq", "dk"):
        assert _qbwd(d, **{name: None}) == -1 and "required" in ttt.ttt_last_error()
        assert _qbwd(d, **{name: FAKE + 1}) == -1 and "elements" in ttt.ttt_last_error()
    for f in (_qfwd, _qbwd):
        assert f(d, inv_freq=None) == -1 and "inv_freq" in ttt.ttt_last_error()
        assert f(d, wq=FAKE + 4) == -1 and f(d, positions=FAKE + 4) == -1
    assert _qfwd(_qk(ldq=512), yq=FAKE) == -1 and "dense" in ttt.ttt_last_error()
    assert _qbwd(d, ws=None) == -3 and _qbwd(d, ws_bytes=4) == -3
    assert _qfwd(_qk(tokens=0), q=None) == 0 and _qbwd(_qk(tokens=0), q=None, dwq=None, dwk=None) == 0
    n = ctypes.c_size_t(0)
    assert B.lib().ttt_qknorm_workspace_size(ctypes.byref(d), None) == -1


def test_sizes_past_32_bits_are_refused_not_cut():
    for kw in (dict(B=1 << 32), dict(T=1 << 32), dict(H=1 << 32), dict(dk=1 << 32), dict(dv=1 << 32), dict(Hk=1 << 32)):
        with pytest.raises(ValueError, match="32 bits"):
            _desc(**kw)
    for kw in (dict(Hq=1 << 32), dict(Hk=1 << 32), dict(d=1 << 32), dict(period=1 << 32)):
        with pytest.raises(ValueError, match="32 bits"):
            _qk(**kw)
    with pytest.raises(ValueError, match="32 bits"):
        B.ttt_delta_step(_desc(T=1), FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE, FAKE, n_states=1 << 32)


def test_host_tensors_are_refused():
    q = torch.zeros(3, 300, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="q must be on the GPU"):
        B.ttt_delta_fwd(_desc(), q, q, FAKE, FAKE, FAKE, None, None, FAKE, None, None, FAKE)
    with pytest.raises(ValueError, match="q must be on the GPU"):
        B.ttt_qknorm_fwd(_qk(), q[0, :10], q[0, :10], None, None, None, FAKE, FAKE, FAKE)


def test_buffers_take_the_documented_shapes_only():
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    st = torch.tensor([0, 3, 5], dtype=torch.int32)
    d = DeltaBuffers(z(5, 2, 8), z(5, 2, 8), z(5, 4, 16), z(5, 4), z(5, 4), seq_starts=st).desc
    assert (d.B, d.T, d.H, d.Hk, d.dk, d.dv, d.packed) == (2, 5, 4, 2, 8, 16, 1)
    d = DeltaBuffers(z(2, 5, 2, 8), z(2, 5, 2, 8), z(2, 5, 4, 16), None, z(2, 5, 4), with_bwd=True).desc
    assert (d.B, d.T, d.H, d.Hk, d.packed) == (2, 5, 4, 2, 0)
    for q, k, v in ((z(5, 2, 8), z(5, 2, 8), z(5, 4, 16)), (z(2, 5, 2, 8), z(2, 5, 1, 8), z(2, 5, 4, 16)),
                    (z(2, 5, 2, 8), z(2, 5, 2, 8), z(2, 6, 4, 16))):
        with pytest.raises(ValueError, match="q and k must be"):
            DeltaBuffers(q, k, v, None, z(*v.shape[:-1]))
    with pytest.raises(ValueError, match="beta must have shape"):
        DeltaBuffers(z(2, 5, 2, 8), z(2, 5, 2, 8), z(2, 5, 4, 16), None, z(2, 5, 2))
    with pytest.raises(ValueError, match="gate must have shape"):
        DeltaBuffers(z(2, 5, 2, 8), z(2, 5, 2, 8), z(2, 5, 4, 16), z(2, 4, 5), z(2, 5, 4))
    whole = z(2, 5, 64)
    q, k, v = whole[..., :16].unflatten(-1, (2, 8)), whole[..., 16:32].unflatten(-1, (2, 8)), whole[..., 32:].unflatten(-1, (4, 8))
    d = DeltaBuffers(q, k, v, None, z(2, 5, 4), with_bwd=True)
    assert (d.desc.ldq, d.desc.ldk, d.desc.ldv) == (64, 64, 64) and d.dq.stride() == q.stride()
    with pytest.raises(ValueError, match="side by side"):
        DeltaBuffers(q, k, whole[..., ::2].unflatten(-1, (4, 8)), None, z(2, 5, 4))
    n = QkNormBuffers(q, k, inv_freq=torch.zeros(3), with_bwd=True)
    assert (n.desc.tokens, n.desc.Hq, n.desc.Hk, n.desc.d, n.desc.rot, n.desc.ldq) == (10, 2, 2, 8, 6, 64)
    for q_, k_ in ((q, k[:1]), (z(5, 8), z(5, 8)), (q, z(2, 5, 2, 4))):
        with pytest.raises(ValueError, match="q and k must be"):
            QkNormBuffers(q_, k_)
