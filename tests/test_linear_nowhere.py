"""A matrix without values overlaps nothing, wherever its pointer points."""
from __future__ import annotations

import pytest
import torch

import trellis_coded_row_amd as cp


@pytest.mark.gpu
def test_inputs_of_no_columns():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    stream = torch.cuda.current_stream().cuda_stream
    y = torch.full((5, 7), 3.0, device="cuda")
    inside = y.data_ptr() + 40
    assert cp.cp_linear(inside, 7, inside, 7, None, None, 0, cp.CP_DTYPE_F32, 5, 7, 0, 0, 0.0, None, y.data_ptr(), 7, None, None, 0,
                        stream) == cp.CP_OK
    assert (y == 0).all()
    assert cp.cp_linear_dx(inside, 0, inside, 7, None, 0, cp.CP_DTYPE_F32, 5, 0, 7, y.fill_(3.0).data_ptr(), None, 0, stream) == cp.CP_OK
    assert (y == 0).all()
    assert cp.cp_linear_dw(inside, 5, inside, 7, cp.CP_DTYPE_F32, 0, 5, 7, 0, y.fill_(3.0).data_ptr(), 7, None, 0, stream) == cp.CP_OK
    assert (y == 0).all()
