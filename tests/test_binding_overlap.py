"""The binding's check that a call's outputs share no memory with what it reads (no GPU needed)."""
import pytest
import torch

from test_ridge_regression_b200 import gka


def test_spans_of_strided_tensors():
    wide = torch.zeros(2, 8, 12, 64, dtype=torch.bfloat16)
    z = wide[:, :, :4]   # its rows lie 12 heads apart: 4 of y's fit in between
    last = 1 * 8 * 12 * 64 + 7 * 12 * 64 + 3 * 64 + 63
    flat = wide.view(-1)
    for start in (0, 4 * 64, last - 5, last):
        with pytest.raises(ValueError):
            gka._apart(z, flat[start:start + 64])
    gka._apart(z, flat[last + 1:last + 65])
    gka._apart(wide[:1], wide[1:])
    gka._apart(z, None)
    gka._apart(wide[:, :0], flat[:64])
    with pytest.raises(ValueError):
        gka._apart(wide[:1], flat[100:200])
    with pytest.raises(ValueError):
        gka._apart(z, z)
