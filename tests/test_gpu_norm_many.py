"""RMS norm of more rows than workgroups stay for: each goes through several
rows and reads one ahead. Tolerances as in test_gpu_norm.py."""
from __future__ import annotations

import pytest
import torch

import trellis_coded_row_amd as cp
from ops_reference import HALF

pytestmark = pytest.mark.gpu
SUM = 52 * 2.0**-24
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    torch.cuda.init()


@pytest.mark.parametrize("n,d", [(9001, 64), (4500, 1000), (2500, 2000), (2300, 4090), (1300, 8192), (600, 12_000),
                                 (700, 24_576), (300, 32_000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(n, d, dtype, residual):
    print(f"norm n={n} d={d} {dtype} residual={residual}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(n + d)
    x = torch.randn(n, d + 3, device="cuda", generator=g).to(dtype)[:, :d]  # rows that start anywhere
    r = torch.randn(n, d, device="cuda", generator=g).to(dtype) if residual else None
    w = (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(dtype)
    x[n // 2] = 0
    out = cp.rms_norm(x, w, residual=r, eps=EPS, fp8=True, rstd=True)
    h = x.double() + (r.double() if residual else 0)
    rstd = 1 / torch.sqrt((h * h).mean(1) + EPS)
    y = h * rstd[:, None] * w.double()
    slack = y.abs() * (SUM + 4 * 2.0**-24)
    assert ((out.rstd.double() - rstd).abs() <= rstd * SUM).all()
    assert ((out.y.double() - y).abs() <= y.abs() * HALF[dtype] + slack + 2.0**-25).all()
    if residual:
        assert ((out.h.double() - h).abs() <= h.abs() * (HALF[dtype] + 2.0**-24) + 2.0**-25).all()
    scale = out.scale.double()
    wide = scale.repeat_interleave(128, 1)[:, :d]
    v = y / wide
    half = torch.maximum(v.abs() * 2.0**-4, torch.full_like(v, 2.0**-10))
    assert ((out.q.double() - v).abs() <= half + slack / wide).all()
    top = torch.nn.functional.pad(y.abs(), (0, -d % 128)).view(n, -1, 128).amax(2)
    edge = 1 + SUM + 4 * 2.0**-24
    assert (top <= 448 * scale * edge).all()  # large enough, and the least such
    assert ((top * edge > 224 * scale) | ((top == 0) & (scale == 1))).all()
    # a row's results do not depend on the rows about it
    again = cp.rms_norm(x.flip(0), w, residual=None if r is None else r.flip(0), eps=EPS, fp8=True, rstd=True)
    assert torch.equal(again.y.flip(0), out.y) and torch.equal(again.rstd.flip(0), out.rstd)
    assert torch.equal(again.q.view(torch.uint8).flip(0), out.q.view(torch.uint8))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_values_that_are_not_finite_stay_in_their_rows(dtype):
    n, d = 3000, 2048
    x = torch.randn(n, d, device="cuda").to(dtype)
    w = torch.ones(d, dtype=dtype, device="cuda")
    want = cp.rms_norm(x, w, fp8=True)
    x[1500, 5], x[2999, 2047] = float("inf"), float("nan")
    out = cp.rms_norm(x, w, fp8=True)
    rows = torch.ones(n, dtype=torch.bool, device="cuda")
    rows[[1500, 2999]] = False
    assert torch.equal(out.y[rows], want.y[rows])
    assert torch.equal(out.q.view(torch.uint8)[rows], want.q.view(torch.uint8)[rows])
    assert torch.isnan(out.q[2999].float()).all() and torch.isnan(out.q[1500, 5].float())
    assert (out.q[1500].float().nan_to_num() == 0).all()
