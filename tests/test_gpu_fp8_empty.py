"""The 8-bit product of matrices without columns or rows, from whatever made them."""
from __future__ import annotations

import pytest
import torch

import trellis_coded_row_amd as cp

pytestmark = pytest.mark.gpu
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    torch.cuda.init()


@pytest.mark.parametrize("m,n", [(5, 7), (1, 300), (200, 1), (0, 4), (4, 0), (0, 0)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_no_columns(m, n, dtype):
    made = lambda rows, kind: torch.empty(rows, 0, dtype=kind, device="cuda")
    quantised = [cp.quantize_fp8(torch.empty(rows, 0, device="cuda"))[:2] for rows in (m, n)]
    for a, sa, b, sb in ((made(m, E4M3), made(m, E8M0), made(n, E4M3), made(n, E8M0)), (*quantised[0], *quantised[1]),
                         (made(m, E4M3), made(m, E8M0), made(n, E4M3), made(-(-n // 128), E8M0))):
        out = cp.gemm_fp8(a, sa, b, sb, dtype=dtype)
        assert out.shape == (m, n) and (out == 0).all()
        into = torch.full((m, n), 3.0, dtype=dtype, device="cuda")
        assert (cp.gemm_fp8(a, sa, b, sb, dtype=dtype, out=into) == 0).all()


@pytest.mark.parametrize("m,n", [(0, 4), (4, 0), (0, 0)])
def test_no_rows(m, n):
    a, sa, _, _ = cp.quantize_fp8(torch.ones(m, 200, device="cuda"))
    b, sb, _, _ = cp.quantize_fp8(torch.ones(n, 200, device="cuda"))
    assert cp.gemm_fp8(a, sa, b, sb).shape == (m, n)
    plain = torch.empty(m, 200, dtype=E4M3, device="cuda"), torch.empty(m, 2, dtype=E8M0, device="cuda")
    if m == 0:
        assert cp.gemm_fp8(*plain, b, sb).shape == (m, n)
