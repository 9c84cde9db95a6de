"""The gradient of the product's epilogue without rows: db is still written, so its workspace and its place are checked."""
from __future__ import annotations

import pytest
import torch

import trellis_coded_row_amd as cp

E = cp.CP_ERR_INVALID_ARGUMENT
R, T, WS = (1 << k for k in (41, 42, 47))  # stand-in addresses, never dereferenced: every call below ends in its checks


def grad(n, db=R, p=0.0, rng=None, ws=WS, wb=1 << 40, dtype=cp.CP_DTYPE_BF16):
    return cp.cp_linear_act_grad(None, n, None, n, dtype, 0, n, cp.CP_ACT_SILU, p, rng, None, db, ws, wb, None)


@pytest.mark.parametrize("n", [1, 64, 1030, 20000])
def test_sums_of_no_rows_need_their_workspace(n):
    need = cp.cp_linear_act_grad_workspace_bytes(0, n)
    assert need >= 4 * n
    for dtype in (cp.CP_DTYPE_F32, cp.CP_DTYPE_BF16, cp.CP_DTYPE_F16):
        assert grad(n, ws=None, dtype=dtype) == E and grad(n, ws=None, wb=0, dtype=dtype) == E
        assert grad(n, wb=need - 1, dtype=dtype) == E and grad(n, ws=WS + 128, dtype=dtype) == E
        assert grad(n, db=None, ws=None, wb=0, dtype=dtype) == cp.CP_OK


def test_sums_of_no_rows_stay_off_the_random_numbers():
    assert grad(64, db=T, p=0.5, rng=T) == E and grad(64, db=T - 4 * 63, p=0.5, rng=T) == E
    assert grad(64, p=0.5, rng=None) == E and grad(64, db=R + 2) == E


@pytest.mark.gpu
def test_sums_of_no_rows_are_zeros():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    stream = torch.cuda.current_stream().cuda_stream
    rng = torch.tensor([1, 2], device="cuda")
    for n in (1, 64, 1030, 20000):
        need = cp.cp_linear_act_grad_workspace_bytes(0, n)
        for dtype in (cp.CP_DTYPE_F32, cp.CP_DTYPE_BF16, cp.CP_DTYPE_F16):
            for act, p in ((cp.CP_ACT_NONE, 0.0), (cp.CP_ACT_GELU, 0.5)):
                ws = torch.full((need + 256,), 0x7F, dtype=torch.uint8, device="cuda")
                db = torch.full((n + 2,), 5.0, device="cuda")
                assert cp.cp_linear_act_grad(None, n, None, n, dtype, 0, n, act, p, rng.data_ptr() if p else None, None,
                                             db.data_ptr() + 4, ws.data_ptr(), need, stream) == cp.CP_OK
                assert db[0] == 5 and db[-1] == 5 and (db[1:-1] == 0).all() and (ws[need:] == 0x7F).all()
