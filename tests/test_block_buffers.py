"""What the recurrence's and the layer norm's buffers make of their tensors (CPU: nothing is launched)."""
import pytest
import torch

from chunkwise_weight_recurrence_amd.layer import LayerNormBuffers, RecurrenceBuffers


def _zeros(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_recurrence_takes_the_documented_shapes_only():
    starts = torch.tensor([0, 3, 5], dtype=torch.int32)
    d = RecurrenceBuffers(_zeros(5, 8), _zeros(5, 8), seq_starts=starts).desc
    assert (d.B, d.T, d.D, d.packed) == (2, 5, 8, 1)
    d = RecurrenceBuffers(_zeros(2, 5, 8), _zeros(2, 5, 8)).desc
    assert (d.B, d.T, d.D, d.packed) == (2, 5, 8, 0)
    # a batch axis in front of packed rows would be taken for the tokens, a head axis too
    for shape, st in (((1, 5, 8), starts), ((5,), starts), ((2, 3, 5, 8), None), ((5, 8), None), ((5, 1), None)):
        with pytest.raises(ValueError, match=r"x must be \["):
            RecurrenceBuffers(_zeros(*shape), _zeros(*shape), seq_starts=st)
    # a longer gate has other tokens' rows from the second sequence on
    RecurrenceBuffers(_zeros(2, 5, 8), _zeros(10, 8))   # the same rows
    with pytest.raises(ValueError, match="gate must have x's shape"):
        RecurrenceBuffers(_zeros(2, 5, 8), _zeros(2, 6, 8))


def test_layer_norm_takes_a_residual_of_its_own_shape_only():
    with pytest.raises(ValueError, match="res must have x's shape"):
        LayerNormBuffers(_zeros(2, 5, 8), res=_zeros(2, 6, 8))
    for shape in ((2, 5, 8), (10, 8)):
        assert LayerNormBuffers(_zeros(2, 5, 8), res=_zeros(*shape)).desc.rows == 10


def test_the_row_distance_of_any_strided_view():
    wide = _zeros(3, 6, 40)
    for rows, ld in ((wide[..., :16], 40), (wide[:, :1, :16], 240), (wide[:, 5:, 8:24], 240), (wide[1:2, :, :16], 40),
                     (wide[1:2, 3:4, :16], 16), (wide[:, ::2, :16], 80), (wide[:, :0, :16], 16), (_zeros(3, 1, 16), 16)):
        buf = RecurrenceBuffers(rows, rows, with_bwd=True)
        assert (buf.desc.ldx, buf.desc.ldg) == (ld, ld) and buf.dx.stride() == rows.stride() == buf.dgate.stride()
        norm = LayerNormBuffers(rows, with_bwd=True)
        assert norm.desc.ldx == ld and norm.dx.stride() == rows.stride()
    d = RecurrenceBuffers(wide[:, :1, :16], _zeros(3, 1, 16)).desc   # one of them strided
    assert (d.ldx, d.ldg) == (240, 16)
    assert LayerNormBuffers(_zeros(16)).desc.ldx == 16 and LayerNormBuffers(wide[0, :, :16]).desc.ldx == 40
