"""The 8-bit product at the sizes that its largest tiles take: ends inside a
tile, a step and a chunk of 16 values, one step, odd numbers of steps, and
splits of k; and its few-row kernel over many and few steps."""
from __future__ import annotations

import pytest
import torch

import trellis_coded_row_amd as cp

from ops_reference import HALF, groups

pytestmark = pytest.mark.gpu
SIZES = [(3000, 4100, 300), (2100, 4000, 100), (2300, 4100, 17), (4100, 4000, 1), (4100, 4000, 390), (2048, 4096, 1100),
         (4096, 4096, 1152), (4000, 4200, 1288), (2048, 2048, 24576), (1024, 1030, 24500)]
ROWS = [(1, 40, 24576), (8, 4096, 1000), (16, 100, 4097), (17, 130, 8192), (32, 4000, 520), (33, 50, 24500), (64, 64, 130)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    torch.cuda.init()


def poisoned(t, unit, byte):
    """t with `byte` in its rows' bytes past their end."""
    if t.shape[1] % unit:
        whole = t.as_strided((t.shape[0], t.shape[1] + -t.shape[1] % unit), (t.stride(0), 1)).view(torch.uint8)
        whole[:, t.shape[1]:] = byte
    return t


def operands(m, n, k, blocks):
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    x = torch.randn(m, k, device="cuda", generator=g) * torch.exp(torch.randn(m, 1, device="cuda", generator=g))
    y = torch.randn(n, k, device="cuda", generator=g) * torch.exp(torch.randn(n, 1, device="cuda", generator=g))
    a, sa, _, _ = cp.quantize_fp8(x)
    b, sb, _, _ = cp.quantize_fp8(y, blocks=blocks)
    return poisoned(a, 16, 0x7F), poisoned(sa, 4, 0xFF), poisoned(b, 16, 0x7F), poisoned(sb, 4, 0xFF)


@pytest.mark.parametrize("m,n,k", SIZES + ROWS)
@pytest.mark.parametrize("blocks", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product(m, n, k, blocks, dtype):
    print(f"tiles m={m} n={n} k={k} blocks={blocks} {dtype}", flush=True)
    a, sa, b, sb = operands(m, n, k, blocks)
    out = cp.gemm_fp8(a, sa, b, sb, dtype=dtype)
    x = a.double() * sa.double().repeat_interleave(128, 1)[:, :k]
    sy = sb.double().repeat_interleave(128, 0)[:n] if blocks else sb.double()
    y = b.double() * sy.repeat_interleave(128, 1)[:, :k]
    want, mags = x @ y.t(), x.abs() @ y.abs().t()
    tol = mags * (k + 2) * 2.0**-24  # a sum of k products in 32 bits
    if dtype != torch.float32:  # products cut off 2^-15 below a group's largest, and the output's rounding
        tol = tol + mags * 2.0**-13 + want.abs() * HALF[dtype] + 2.0**-25
    bad = ~((out.double() - want).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, first at {torch.nonzero(bad)[0].tolist()}"
    assert torch.equal(out, cp.gemm_fp8(a, sa, b, sb, dtype=dtype))


@pytest.mark.parametrize("m,n,k", [(3000, 4100, 300), (4100, 4000, 520), (2100, 4000, 100)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_place_is_multiplied_once(m, n, k, dtype):
    # one-hot rows: out[i][j] = a[i][p_i] b[j][p_i], exact in every type
    print(f"one-hot m={m} n={n} k={k} {dtype}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(k)
    p = torch.randint(0, k, (m,), device="cuda", generator=g)
    x = torch.zeros(m, k + -k % 16, device="cuda")
    x[torch.arange(m, device="cuda"), p] = torch.randint(1, 8, (m,), device="cuda", generator=g).float()
    y = torch.zeros(n, k + -k % 16, device="cuda")
    y[:, :k] = torch.randint(-8, 9, (n, k), device="cuda", generator=g).float()
    one = lambda rows: torch.full((rows, groups(k) + -groups(k) % 4), 127, dtype=torch.uint8, device="cuda").view(
        torch.float8_e8m0fnu)[:, :groups(k)]
    out = cp.gemm_fp8(x.to(torch.float8_e4m3fn)[:, :k], one(m), y.to(torch.float8_e4m3fn)[:, :k], one(n), dtype=dtype)
    assert torch.equal(out.float(), x[torch.arange(m, device="cuda"), p][:, None] * y.t()[p])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_what_is_not_a_number_stays_in_its_row_and_column(dtype):
    m, n, k = 3000, 4100, 300
    a, sa, b, sb = operands(m, n, k, False)
    a.view(torch.uint8)[2999, 299] = 0x7F
    sb.view(torch.uint8)[4000, 1] = 0xFF
    out = cp.gemm_fp8(a, sa, b, sb, dtype=dtype)
    assert torch.isnan(out[2999]).all() and torch.isnan(out[:, 4000]).all()
    rows, cols = torch.arange(m, device="cuda") != 2999, torch.arange(n, device="cuda") != 4000
    assert torch.isfinite(out[rows][:, cols]).all()
