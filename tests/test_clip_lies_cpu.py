"""How gradients that are no dense tensors lie, for the clipping call (CPU only)."""

import pytest
import torch

from matrix_roots_amd import binding as B


def test_columns_are_rows_of_one_value():
    big = torch.zeros(6, 10, 16)
    for t, want in [(big[0, :, :1], (10, 1, 16)), (big[0, :, 7:8], (10, 1, 16)), (big[:, :, 3:4], (60, 1, 16)),
                    (big[:, 2:3, 5:6], (6, 1, 160)), (big[0, :, :1].t(), (10, 1, 16)), (big[0, 2:3, :5], (1, 5, 0)),
                    (big[:, :1, :5], (6, 5, 160))]:
        assert B._rows_of(t) == want, (t.shape, t.stride())
    # values further apart in rows of more than one are no rows, nor are vectors with a stride
    for t in (big[0, :, ::2], big[0, 0, ::2], torch.zeros(1, 1).expand(5, 1), torch.zeros(1, 8).expand(4, 8)):
        with pytest.raises(ValueError):
            B._rows_of(t)


def test_columns_and_dense_outputs():
    big = torch.zeros(6, 16)
    assert B._clip_lies(0, big[:, 4:5], torch.zeros(6, 1)) == (6, 1, 16, 1)
    assert B._clip_lies(0, big[:, 4:5], big[:, 5:6]) == (6, 1, 16, 16)
    assert B._clip_lies(0, big[:, 4:5], None) == (6, 1, 16, 16)


def test_strides_of_single_values_do_not_matter():
    """A dimension of one value may have any stride: the tensors lie alike all the same."""
    a, b = torch.zeros(5, 14, 7)[:, :1], torch.zeros(5, 98).as_strided((5, 1, 7), (98, 98, 1))
    assert a.stride() != b.stride()
    assert B._clip_lies(0, a, b) == (5, 7, 98, 98)
    with pytest.raises(ValueError):
        B._clip_lies(0, a, torch.zeros(5, 1, 7))
