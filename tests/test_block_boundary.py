"""Refusals of the recurrence and layer norm entry points (CPU): bad arguments are
rejected on the host, before any HIP call, with the documented status."""
import ctypes

import pytest
import torch

import chunkwise_weight_recurrence_amd as ttt
from chunkwise_weight_recurrence_amd import binding as B

FAKE = 0x1000   # never dereferenced: every case below fails validation first or has nothing to do


@pytest.fixture(scope="module")
def L():
    return B.lib()


def _rec(**kw):
    base = dict(B=3, T=300, D=64)
    base.update(kw)
    return B.make_rec_desc(**base)


def _fwd(d, **kw):
    p = dict(x=FAKE, gate=FAKE, h0=None, seq_starts=None, o=FAKE, h_final=None, saved=None, ws=FAKE, ws_bytes=1 << 30)
    p.update(kw)
    return B.lib().ttt_recurrence_fwd(ctypes.byref(d) if d is not None else None, *p.values(), None)


def _bwd(d, **kw):
    p = dict(x=FAKE, gate=FAKE, h0=None, seq_starts=None, saved=FAKE, d_o=FAKE, d_hfinal=None, dx=FAKE, dgate=FAKE,
             dh0=None, ws=FAKE, ws_bytes=1 << 30)
    p.update(kw)
    return B.lib().ttt_recurrence_bwd(ctypes.byref(d), *p.values(), None)


def _step(d, **kw):
    p = dict(x=FAKE, gate=FAKE, slots=None, n_states=3, h=FAKE, o=FAKE)
    p.update(kw)
    return B.lib().ttt_recurrence_step(ctypes.byref(d), *p.values(), None)


def test_struct_sizes():
    assert ctypes.sizeof(B.TTTRecDesc) == 48 and ctypes.sizeof(B.TTTLnDesc) == 40


def test_enums_match_header():
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ttt.h")).read()
    for cls, prefix in ((B.Gate, "TTT_GATE_"), (B.RecInput, "TTT_REC_")):
        for m in cls:
            assert int(re.search(rf"\b{prefix}{m.name}\s*=\s*(\d+)", src).group(1)) == int(m)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(B=-1), -1, "B, T"), (dict(T=-1), -1, "B, T"), (dict(D=0), -1, "D must be"), (dict(packed=2), -1, "packed"),
    (dict(dtype=7), -1, "dtype"), (dict(gate=2), -1, "gate"), (dict(input=-1), -1, "input"),
    (dict(ldx=63), -1, "ldx, ldg"), (dict(ldg=1), -1, "ldx, ldg"), (dict(ldx=-64), -1, "ldx, ldg"),
    (dict(B=1 << 16, T=1 << 15), -2, "too large"), (dict(D=(1 << 24) + 1), -2, "too large"),
    (dict(ldx=1 << 40), -2, "too large"), (dict(B=1, T=2_000_000_000, D=1 << 20), -2, "too large"),
    # a launch has fewer than 2^32 threads
    (dict(B=1, T=(1 << 30) - 127, D=64), -2, "too large"), (dict(B=1 << 20, T=1, D=(1 << 16) + 64), -2, "too large"),
])
def test_recurrence_desc(L, kw, code, msg):
    d = _rec(**kw)
    n = ctypes.c_size_t(0)
    for st in (_fwd(d), _bwd(d), _step(d), L.ttt_recurrence_workspace_size(ctypes.byref(d), 0, ctypes.byref(n)),
               L.ttt_recurrence_saved_size(ctypes.byref(d), ctypes.byref(n))):
        assert st == code and msg in ttt.ttt_last_error()


@pytest.mark.parametrize("kw", [
    dict(B=(1 << 31) - 1, packed=True), dict(B=(1 << 31) - 4095, packed=True, D=1), dict(B=(1 << 31) - 4095, T=0, D=1),
    dict(B=1 << 30, T=0, D=1 << 13), dict(B=1 << 30, D=1 << 13, packed=True),
])
def test_recurrence_sequence_count(L, kw):
    """Sequences without a token are no tokens, but they are indexed in 32 bits as those are."""
    d, n = _rec(**kw), ctypes.c_size_t(0)
    p = dict(seq_starts=FAKE) if d.packed else {}
    for st in (_fwd(d, **p), _bwd(d, **p), L.ttt_recurrence_workspace_size(ctypes.byref(d), 0, ctypes.byref(n)),
               L.ttt_recurrence_saved_size(ctypes.byref(d), ctypes.byref(n))):
        assert st == -2 and "too large" in ttt.ttt_last_error()
    assert _fwd(_rec(B=(1 << 31) - 4096, T=0, D=1)) == 0   # without h_final there is nothing to launch


def test_recurrence_pointers_and_workspace(L):
    d, p = _rec(), _rec(packed=True)
    assert _fwd(None) == -1 and "desc is NULL" in ttt.ttt_last_error()
    for name in ("x", "gate", "o"):
        assert _fwd(d, **{name: None}) == -1 and "required" in ttt.ttt_last_error()
    for name in ("x", "gate", "saved", "d_o", "dx", "dgate"):
        assert _bwd(d, **{name: None}) == -1 and "required" in ttt.ttt_last_error()
    for f in (_fwd, _bwd):
        assert f(p) == -1 and "seq_starts" in ttt.ttt_last_error()
        assert f(d, seq_starts=FAKE) == -1 and "seq_starts" in ttt.ttt_last_error()
        assert f(d, x=FAKE + 2) == -1 and "x must be 16-byte aligned" in ttt.ttt_last_error()
        assert f(d, ws=None) == -3 and f(d, ws_bytes=16) == -3
    assert _fwd(p, seq_starts=FAKE + 4) == -1 and "seq_starts must be 16-byte" in ttt.ttt_last_error()
    # the state that a call reads may not be the one that it writes, not even in part
    assert _fwd(d, h0=FAKE, h_final=FAKE) == -1 and "overlap" in ttt.ttt_last_error()
    assert _fwd(d, h0=FAKE, h_final=FAKE + 3 * 64 * 4 - 16) == -1
    assert _bwd(d, d_hfinal=FAKE + 16, dh0=FAKE) == -1 and "overlap" in ttt.ttt_last_error()
    assert L.ttt_recurrence_workspace_size(ctypes.byref(d), 2, ctypes.byref(ctypes.c_size_t(0))) == -1
    assert L.ttt_recurrence_workspace_size(ctypes.byref(d), 0, None) == -1


def test_recurrence_sizes():
    assert ttt.ttt_recurrence_workspace_size(_rec(B=1, T=100), 0) == 0   # one run of tokens needs no exchange
    assert ttt.ttt_recurrence_workspace_size(_rec(), 0) > 0
    assert ttt.ttt_recurrence_saved_size(_rec()) >= 8 * 64 * 4           # 900 tokens: 8 runs of 128


def test_recurrence_empty_problems_need_no_device():
    none = dict(x=None, gate=None, o=None, ws=None, ws_bytes=0)
    assert _fwd(_rec(B=0, T=0), **none) == 0 and _fwd(_rec(T=0), **none) == 0
    assert _fwd(_rec(B=0, T=0, packed=True), **none) == 0
    assert _bwd(_rec(T=0), x=None, gate=None, saved=None, d_o=None, dx=None, dgate=None) == 0
    assert _step(_rec(B=0, T=1), x=None, h=None) == 0


def test_step_refusals():
    d = _rec(T=1)
    assert _step(_rec(T=2)) == -1 and "T = 1" in ttt.ttt_last_error()
    assert _step(_rec(T=1, packed=True)) == -1
    assert _step(d, n_states=2) == -1 and "n_states" in ttt.ttt_last_error()   # three rows without slots
    assert _step(d, n_states=-1) == -1
    assert _step(_rec(B=1 << 24, T=1), n_states=1 << 24) == -2 and "too large" in ttt.ttt_last_error()
    for name in ("x", "gate", "h", "o"):
        assert _step(d, **{name: None}) == -1 and "required" in ttt.ttt_last_error()
    assert _step(d, h=FAKE + 8) == -1 and "h must be 16-byte aligned" in ttt.ttt_last_error()


def test_step_with_slots_is_bounded():
    """Each row looks for its slot among all others: millions of rows would hold the GPU for minutes."""
    n = (1 << 20) + 1
    assert _step(_rec(B=n, T=1), slots=FAKE) == -2 and "too large" in ttt.ttt_last_error()
    assert _step(_rec(B=n - 1, T=1), slots=FAKE, x=None) == -1 and "required" in ttt.ttt_last_error()
    assert _step(_rec(B=n, T=1), n_states=n, x=None) == -1 and "required" in ttt.ttt_last_error()   # without slots


def _ln(**kw):
    base = dict(rows=12, D=64)
    base.update(kw)
    return B.make_ln_desc(**base)


def _lfwd(d, **kw):
    p = dict(x=FAKE, res=None, w=FAKE, b=FAKE, y=FAKE, r=None, mean=None, rstd=None)
    p.update(kw)
    return B.lib().ttt_layernorm_fwd(ctypes.byref(d) if d is not None else None, *p.values(), None)


def _lbwd(d, **kw):
    p = dict(x=FAKE, w=FAKE, mean=FAKE, rstd=FAKE, dy=FAKE, dr=None, dx=FAKE, dw=FAKE, db=FAKE, ws=FAKE,
             ws_bytes=1 << 30)
    p.update(kw)
    return B.lib().ttt_layernorm_bwd(ctypes.byref(d), *p.values(), None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(rows=-1), -1, "rows"), (dict(D=0), -1, "D must be"), (dict(groups=0), -1, "groups"),
    (dict(period=0), -1, "groups"), (dict(groups=5), -1, "multiple"), (dict(groups=3, period=5), -1, "multiple"),
    (dict(dtype=3), -1, "dtype"), (dict(eps=-1.0), -1, "eps"), (dict(eps=float("nan")), -1, "eps"),
    (dict(ldx=60), -1, "ldx"), (dict(rows=1 << 31), -2, "too large"), (dict(D=(1 << 24) + 1), -2, "too large"),
])
def test_layernorm_desc(L, kw, code, msg):
    d = _ln(**kw)
    for st in (_lfwd(d), _lbwd(d), L.ttt_layernorm_workspace_size(ctypes.byref(d), ctypes.byref(ctypes.c_size_t(0)))):
        assert st == code and msg in ttt.ttt_last_error()


def test_layernorm_pointers_and_workspace():
    d = _ln()
    assert _lfwd(None) == -1 and "desc is NULL" in ttt.ttt_last_error()
    assert _lfwd(d, x=None) == -1 and _lfwd(d, y=None) == -1 and "required" in ttt.ttt_last_error()
    assert _lfwd(d, res=FAKE) == -1 and "go together" in ttt.ttt_last_error()
    assert _lfwd(d, r=FAKE) == -1
    assert _lfwd(d, w=FAKE + 4) == -1 and "w must be 16-byte aligned" in ttt.ttt_last_error()
    for name in ("x", "mean", "rstd", "dy", "dx"):
        assert _lbwd(d, **{name: None}) == -1 and "required" in ttt.ttt_last_error()
    assert _lbwd(d, ws=None) == -3 and _lbwd(d, ws_bytes=16) == -3
    assert _lfwd(_ln(rows=0), x=None, y=None) == 0
    assert _lbwd(_ln(rows=0), x=None, mean=None, rstd=None, dy=None, dx=None, dw=None, db=None, ws=None) == 0


def test_binding_refuses_tensors_that_would_fault():
    d, x = _rec(B=1, T=8, D=4), torch.zeros(1, 8, 4, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x must be on the GPU"):
        ttt.ttt_recurrence_fwd(d, x, x, None, None, x, None, None, None)
    with pytest.raises(ValueError, match="x must be on the GPU"):
        ttt.ttt_layernorm_fwd(_ln(), x, None, None, None, x, None, None, None)
    with pytest.raises(TypeError):
        ttt.ttt_recurrence_fwd(d, [1], x, None, None, x, None, None, None)

    class Fake:  # a tensor that says it is on the GPU
        def __init__(self, t, device="cuda:0"):
            self.t, self.device = t, torch.device(device)

        def get_device(self):
            return self.device.index

        def __getattr__(self, name):
            return getattr(self.t, name)

    f = Fake
    with pytest.raises(ValueError, match="x must be bfloat16, not float32"):
        ttt.ttt_recurrence_fwd(d, f(x.float()), f(x), None, None, f(x), None, None, None)
    with pytest.raises(ValueError, match="gate has 28 elements, 32 are needed"):
        ttt.ttt_recurrence_fwd(d, f(x), f(x[:, 1:]), None, None, f(x), None, None, None)
    with pytest.raises(ValueError, match="gate must be contiguous"):
        ttt.ttt_recurrence_fwd(d, f(x), f(torch.zeros(1, 8, 8, dtype=torch.bfloat16)[..., :4]), None, None, f(x), None, None, None)
    with pytest.raises(ValueError, match="gate must have rows of 4 elements, 9 apart"):
        ttt.ttt_recurrence_fwd(B.make_rec_desc(1, 8, 4, ldg=9), f(x), f(torch.zeros(1, 8, 8, dtype=torch.bfloat16)[..., :4]), None,
                               None, f(x), None, None, None)
    with pytest.raises(ValueError, match="o is on cuda:1, the tensors before it on cuda:0"):
        ttt.ttt_recurrence_fwd(d, f(x), f(x), None, None, f(x, "cuda:1"), None, None, None)
    with pytest.raises(ValueError, match="h has 8 elements"):
        ttt.ttt_recurrence_step(B.make_rec_desc(8, 1, 4), f(x), f(x), None, f(torch.zeros(2, 4)), f(x), n_states=8)
    with pytest.raises(ValueError, match="w has 64 elements, 128 are needed"):
        y = torch.zeros(12, 64, dtype=torch.bfloat16)
        ttt.ttt_layernorm_fwd(_ln(groups=2), f(y), None, f(torch.zeros(64)), None, f(y), None, None, None)


def test_sizes_past_32_bits_are_refused_not_cut():
    """A field of a descriptor would keep the low 32 bits: 2^32 + 128 tokens were 128."""
    big = (1 << 32) + 128
    for name in ("B", "T", "D"):
        with pytest.raises(ValueError, match=f"{name} must fit in 32 bits"):
            _rec(**{name: big})
    for name in ("D", "groups", "period"):
        with pytest.raises(ValueError, match=f"{name} must fit in 32 bits"):
            _ln(**{name: big})
    with pytest.raises(ValueError, match="T must fit in 32 bits"):
        _rec(T=-(1 << 32))
    assert _ln(rows=big).rows == big
    with pytest.raises(ValueError, match="n_states must fit in 32 bits"):
        ttt.ttt_recurrence_step(_rec(T=1), FAKE, FAKE, None, FAKE, FAKE, n_states=(1 << 32) + 3)
