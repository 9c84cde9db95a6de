"""Matrices of no columns through the gradient of the product's epilogue: nothing is launched, and no size is divided by."""
from __future__ import annotations

import pytest
import torch

import trellis_coded_row_amd as cp

P, V, R = (1 << k for k in (40, 41, 42))  # stand-in addresses, never dereferenced


@pytest.mark.parametrize("m", [0, 1, 5, 100, 2**31 - 1])
def test_no_workspace_for_no_columns(m):
    assert cp.cp_linear_act_grad_workspace_bytes(m, 0) == 0
    for dtype in (cp.CP_DTYPE_F32, cp.CP_DTYPE_BF16, cp.CP_DTYPE_F16):
        assert cp.cp_linear_act_grad(P, 64, P, 64, dtype, m, 0, cp.CP_ACT_SILU, 0.0, None, V, R, None, 0, None) == cp.CP_OK


@pytest.mark.gpu
def test_a_gradient_of_no_columns():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    rng = torch.tensor([1, 2], device="cuda")
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        for m in (0, 1, 6, 3000):
            for dy in (torch.ones(m, 0, device="cuda", dtype=dtype), torch.ones(m, 8, device="cuda", dtype=dtype)[:, 8:]):
                for act, p in ((None, 0.0), ("silu", 0.5)):
                    dz, db = cp.linear_act_grad(dy, dy, act=act, p=p, rng=rng)
                    assert dz.shape == (m, 0) and dz.dtype == dtype and db.shape == (0,) and db.dtype == torch.float32
                    dz, db = cp.linear_act_grad(dy, dy, act=act, p=p, rng=rng, db=False)
                    assert dz.shape == (m, 0) and db is None
    torch.cuda.synchronize()
