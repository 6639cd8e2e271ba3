"""What the binding says of logits it does not take: the reason is the right
one (nothing is launched, so host tensors do)."""

import pytest
import torch

from newton_schulz_matrix_amd import operators as ops


def _args(logits):
    labels = torch.zeros(logits.shape[:2], dtype=torch.int64)
    return ops._preference_args(logits, labels, 0.1, 0.0, -1)


def test_layouts_that_are_taken():
    full = torch.zeros(6, 5, 8)
    for logits, ld, sequence in ((full, 8, 0), (full[:, 1:], 8, 40), (full[::3], 8, 120),
                                 (full[..., :7], 8, 40), (full[:2, 2:3], 8, 40)):
        args = _args(logits)
        assert (args.ld, args.ld_sequence) == (ld, sequence)


def test_time_major_logits_are_not_called_overlapping():
    """Positions further apart than sequences: rows of their own, in an order
    that the calls do not take."""
    logits = torch.zeros(5, 6, 8).transpose(0, 1)
    with pytest.raises(ValueError, match="one behind the other") as e:
        _args(logits)
    assert "overlapping" not in str(e.value) and "contiguous()" in str(e.value)


def test_overlapping_rows_are():
    for logits in (torch.zeros(5, 8)[None].expand(4, 5, 8), torch.zeros(4, 1, 8).expand(4, 5, 8),
                   torch.zeros(200).as_strided((4, 5, 8), (20, 8, 1)),
                   torch.zeros(200).as_strided((4, 5, 8), (40, 4, 1)),
                   torch.zeros(200).as_strided((4, 5, 8), (4, 16, 1))):
        with pytest.raises(ValueError, match="overlapping"):
            _args(logits)
