"""RMS norm and its gradient against plain 64-bit forms.

Tolerances: a sum of squares runs through chains of fewer than 96 additions
in 32 bits, so rstd is off by less than 48 + 4 steps of 2^-24 (SUM); y adds
two products and its rounding."""
from __future__ import annotations

import math

import pytest
import torch

import trellis_coded_row_amd as cp
from ops_reference import HALF, on_grid, row_scales, scale_exponent, spread, groups

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]
SUM = 52 * 2.0**-24
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    torch.cuda.init()


def inputs(n, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, d, generator=g) * torch.exp(torch.randn(d, generator=g) * 0.7)
    r = torch.randn(n, d, generator=g)
    w = 1 + 0.2 * torch.randn(d, generator=g)
    return x.to(dtype), r.to(dtype), w.to(dtype)


def check(x, r, w, out, dtype):
    h = x.double() + (r.double() if r is not None else 0)
    rstd = 1 / torch.sqrt((h * h).mean(1) + EPS)
    y = h * rstd[:, None] * w.double()
    slack = y.abs() * (SUM + 4 * 2.0**-24)
    assert ((out.rstd.cpu().double() - rstd).abs() <= rstd * SUM).all()
    if r is not None:
        assert ((out.h.cpu().double() - h).abs() <= h.abs() * (HALF[dtype] + 2.0**-24) + 2.0**-25).all()
    if out.y is not None:
        assert ((out.y.cpu().double() - y).abs() <= y.abs() * HALF[dtype] + slack + 2.0**-25).all()
    if out.q is not None:
        n, d = x.shape
        s = out.scale.cpu().double()
        low, high = row_scales(y * (1 - SUM - 4 * 2.0**-24)), row_scales(y * (1 + SUM + 4 * 2.0**-24))
        assert ((s == low) | (s == high)).all()
        wide = spread(s, n, d)
        got = out.q.cpu().double()
        # half a step of e4m3 about the value (steps of 2^-9 below 2^-6), and the value's own slack
        v = y / wide
        half = torch.maximum(v.abs() * 2.0**-4, torch.full_like(v, 2.0**-10))
        assert ((got - v).abs() <= half + slack / wide).all()
        assert (got == on_grid(got)).all()


SIZES = [(1, 1), (3, 5), (7, 128), (5, 129), (2, 511), (600, 512), (9, 1000), (4, 2048), (3, 2050), (600, 2500),
         (8, 4096), (5, 8190), (600, 5000), (3, 16_000), (2, 24_576), (3, 30_001), (2, 32_768), (2, 40_003)]


@pytest.mark.parametrize("n,d", SIZES)
@pytest.mark.parametrize("dtype", TYPES)
def test_norm(n, d, dtype):
    print(f"norm n={n} d={d} {dtype}", flush=True)
    x, r, w = inputs(n, d, dtype, n + d)
    xc, rc, wc = x.cuda(), r.cuda(), w.cuda()
    out = cp.rms_norm(xc, wc, residual=rc, eps=EPS, y=True, fp8=True, rstd=True)
    check(x, r, w, out, dtype)
    out = cp.rms_norm(xc, wc, eps=EPS, y=False, fp8=True, rstd=True)
    assert out.h is xc and out.y is None
    check(x, None, w, out, dtype)
    out = cp.rms_norm(xc, wc, eps=EPS)
    assert out.q is None and out.scale is None and out.rstd is None and out.y.dtype == dtype


def test_norm_writes_only_its_outputs():
    # a row of 8-bit values that ends before its stride keeps the bytes after it
    n, d = 5, 133
    x, r, w = (t.cuda() for t in inputs(n, d, torch.bfloat16, 1))
    q = torch.full((n, 160), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.full((n, 7), 0x33, dtype=torch.uint8, device="cuda")
    st = cp.cp_rms_norm(x.data_ptr(), d, None, 0, w.data_ptr(), cp.CP_DTYPE_BF16, n, d, EPS, None, None, q.data_ptr(),
                        160, s.data_ptr(), 7, None, torch.cuda.current_stream().cuda_stream)
    assert st == cp.CP_OK
    ref = cp.rms_norm(x, w, eps=EPS, y=False, fp8=True)
    assert (q[:, d:] == 0x5A).all() and (s[:, 2:] == 0x33).all()
    assert (q[:, :d] == ref.q.view(torch.uint8)).all() and (s[:, :2] == ref.scale.view(torch.uint8)).all()


def test_norm_views_zeros_and_values_that_are_not_finite():
    x, _, w = inputs(6, 300, torch.float32, 3)
    big = torch.zeros(6, 1000)
    big[:, 100:400] = x
    out = cp.rms_norm(big.cuda()[:, 100:400], w.cuda(), eps=EPS, fp8=True, rstd=True)
    check(x, None, w, out, torch.float32)
    x[0] = 0
    x[1, 7] = math.inf
    x[2, 8] = math.nan
    out = cp.rms_norm(x.cuda(), w.cuda(), eps=EPS, fp8=True, rstd=True)
    assert (out.y[0] == 0).all() and (out.q[0].float() == 0).all() and (out.scale[0].float() == 1).all()
    assert float(out.rstd[1]) == 0 and torch.isnan(out.y[1, 7]) and (out.y[1, :7] == 0).all()
    assert torch.isnan(out.q[1, 7].float()) and (out.q[1, :7].float() == 0).all()
    assert torch.isnan(out.y[2]).all() and torch.isnan(out.q[2].float()).all()
    assert torch.isfinite(out.y[3:]).all()
    assert cp.rms_norm(torch.empty(0, 16, device="cuda"), torch.ones(16, device="cuda"), fp8=True).q.shape == (0, 16)


def test_norm_refusals():
    x, w = torch.ones(4, 16, device="cuda"), torch.ones(16, device="cuda")
    for call in (lambda: cp.rms_norm(x, w[:8]), lambda: cp.rms_norm(x, w.bfloat16()), lambda: cp.rms_norm(x.t(), w[:4]),
                 lambda: cp.rms_norm(x, w, residual=x[:3]), lambda: cp.rms_norm(x, w, residual=x.half()),
                 lambda: cp.rms_norm(x.long(), w), lambda: cp.rms_norm(x[:, :0], w[:0]),
                 lambda: cp.rms_norm_grad(x, x, torch.ones(3, device="cuda"), w),
                 lambda: cp.rms_norm_grad(x.half(), x, torch.ones(4, device="cuda"), w)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("n,d", SIZES + [(2000, 64), (1111, 1536), (700, 8192)])
@pytest.mark.parametrize("dtype", TYPES)
def test_gradient(n, d, dtype):
    print(f"norm gradient n={n} d={d} {dtype}", flush=True)
    x, dres, w = inputs(n, d, dtype, n * 3 + d)
    dy = torch.randn(n, d, generator=torch.Generator().manual_seed(d)).to(dtype)
    xd, wd, yd = x.double(), w.double(), dy.double()
    rstd = (1 / torch.sqrt((xd * xd).mean(1) + EPS)).float()
    r = rstd.double()[:, None]
    hat, g = xd * r, yd * wd
    mean = (g * hat).mean(1, keepdim=True)
    dx = r * (g - hat * mean)
    # the mean's chain of additions, over the sum of magnitudes; four products of its own
    off = r * (hat.abs() * (g * hat).abs().mean(1, keepdim=True) * 100 + (g.abs() + (hat * mean).abs()) * 6) * 2.0**-24
    dw, dwm = (yd * hat).sum(0), (yd * hat).abs().sum(0)
    for with_res in (True, False):
        gx, gw = cp.rms_norm_grad(dy.cuda(), x.cuda(), rstd.cuda(), w.cuda(), dres=dres.cuda() if with_res else None)
        want = dx + dres.double() if with_res else dx
        assert ((gx.cpu().double() - want).abs() <= off + want.abs() * (HALF[dtype] + 2.0**-23) + 2.0**-25).all()
        # a column's chain: the rows of one group, then the groups' sums
        assert ((gw.cpu().double() - dw).abs() <= dwm * (n + 40) * 2.0**-24).all()


def test_gradient_against_differences():
    g = torch.Generator().manual_seed(2)
    x, w, c = torch.randn(3, 50, generator=g), 1 + 0.1 * torch.randn(50, generator=g), torch.randn(3, 50, generator=g)
    out = cp.rms_norm(x.cuda(), w.cuda(), eps=EPS, rstd=True)
    dx, dw = cp.rms_norm_grad(c.cuda(), x.cuda(), out.rstd, w.cuda())

    def f(x, w):
        x, w = x.double(), w.double()
        return float((c.double() * x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * w).sum())

    step = 1e-5
    for i, k in ((0, 0), (1, 17), (2, 49)):
        e = torch.zeros(3, 50, dtype=torch.float64)
        e[i, k] = step
        slope = (f(x.double() + e, w) - f(x.double() - e, w)) / (2 * step)
        assert abs(slope - float(dx[i, k])) < 1e-5  # the quotient's error step^2, and 32 bits of values near 1
        e = torch.zeros(50, dtype=torch.float64)
        e[k] = step
        slope = (f(x, w.double() + e) - f(x, w.double() - e)) / (2 * step)
        assert abs(slope - float(dw[k])) < 1e-5


def test_gradient_of_nothing_and_of_one_row_for_all():
    w = torch.ones(20, device="cuda")
    dx, dw = cp.rms_norm_grad(torch.empty(0, 20, device="cuda"), torch.empty(0, 20, device="cuda"),
                              torch.empty(0, device="cuda"), w)
    assert dx.shape == (0, 20) and (dw == 0).all()
    x = torch.randn(40, 20, device="cuda")
    rstd = cp.rms_norm(x, w, rstd=True).rstd
    one = torch.randn(1, 20, device="cuda")
    a = cp.rms_norm_grad(one.expand(40, 20), x, rstd, w)
    b = cp.rms_norm_grad(one.expand(40, 20).contiguous(), x, rstd, w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
