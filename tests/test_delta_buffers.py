"""Which states and weights the delta rule's and the query and key norm's buffers take (CPU: nothing is launched)."""
import pytest
import torch

from chunkwise_weight_recurrence_amd.layer import DeltaBuffers, QkNormBuffers


def _z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("packed", [False, True])
def test_delta_states_have_the_rule_s_shape(packed):
    lead, st = ((10,), torch.tensor([0, 4, 10], dtype=torch.int32)) if packed else ((2, 5), None)
    args = (_z(*lead, 2, 8), _z(*lead, 2, 8), _z(*lead, 4, 16), None, _z(*lead, 4))
    f32 = dict(dtype=torch.float32)
    DeltaBuffers(*args, s0=_z(2, 4, 8, 16, **f32), seq_starts=st)
    # as many elements, or more, with the keys' and values' channels, the heads or the sequences elsewhere
    for shape in ((2, 4, 16, 8), (4, 2, 8, 16), (3, 4, 8, 16), (2, 4, 128), (1, 4, 8, 16)):
        with pytest.raises(ValueError, match="s0 must have shape"):
            DeltaBuffers(*args, s0=_z(*shape, **f32), seq_starts=st)
        with pytest.raises(ValueError, match="d_sfinal must have shape"):
            DeltaBuffers(*args, seq_starts=st, with_bwd=True).backward(_z(*lead, 4, 16), _z(*shape, **f32))


def test_query_and_key_weights_have_a_head_s_columns():
    """A weight per head, [H,d], has enough elements too: its first head's would be taken for all."""
    q, k = _z(2, 5, 4, 16), _z(2, 5, 2, 16)
    w = lambda *s: _z(*s, dtype=torch.float32)  # noqa: E731
    QkNormBuffers(q, k, w(16), w(16), with_bwd=True)
    for shape in ((4, 16), (17,), (1, 16), (64,)):
        with pytest.raises(ValueError, match="wq must have shape"):
            QkNormBuffers(q, k, wq=w(*shape))
        with pytest.raises(ValueError, match="wk must have shape"):
            QkNormBuffers(q, k, wk=w(*shape))
    # and one position a token
    pos = lambda *s: _z(*s, dtype=torch.int32)  # noqa: E731
    for ok in (pos(10), pos(2, 5)):
        QkNormBuffers(q, k, positions=ok)
    for bad in (pos(5), pos(11), pos(2, 10)):
        with pytest.raises(ValueError, match="positions must be"):
            QkNormBuffers(q, k, positions=bad)


def test_gradients_of_the_outputs_have_their_heads_and_channels():
    """Heads in front of the tokens, or channels of another tensor, have as many elements."""
    q, v = _z(2, 5, 2, 8), _z(2, 5, 4, 16)
    buf = DeltaBuffers(q, q, v, None, _z(2, 5, 4), with_bwd=True)
    for shape in ((2, 4, 5, 16), (2, 5, 64), (2, 5, 16, 4), (2, 6, 4, 16)):
        with pytest.raises(ValueError, match="d_o must have"):
            buf.backward(_z(*shape))
    norm = QkNormBuffers(_z(2, 5, 4, 16), _z(2, 5, 2, 16), with_bwd=True)
    for dyq, dyk, name in (((2, 4, 5, 16), (2, 5, 2, 16), "dyq"), ((2, 5, 4, 16), (2, 2, 5, 16), "dyk"), ((2, 5, 64), (2, 5, 2, 16), "dyq"),
                           ((2, 5, 4, 16), (1, 5, 4, 16), "dyk")):
        with pytest.raises(ValueError, match=f"{name} must have"):
            norm.backward(_z(*dyq), _z(*dyk))
    # rows of all tokens one behind the other are the same rows: on to the check that they are on the GPU
    with pytest.raises(ValueError, match="GPU"):
        buf.backward(_z(10, 4, 16))
    with pytest.raises(ValueError, match="GPU"):
        norm.backward(_z(10, 4, 16), _z(10, 2, 16))
