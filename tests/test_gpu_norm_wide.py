"""The norm and its gradient at rows of more columns than one launch has
threads for."""
from __future__ import annotations

import pytest
import torch

import trellis_coded_row_amd as cp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    torch.cuda.init()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n,d", [(1, 2**26), (2, 2**27 + 8), (1, 2**28 + 3)])
def test_gradient_of_long_rows(n, d):
    # dw is a sum of n products of two roundings each; dx's mean of d terms is far below its own rounding here: the
    # terms have random signs, so that its sum in 32 bits is off by at most d^1/2 steps of 2^-24 of d^1/2
    print(f"gradient n={n} d={d}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(n)
    x, dy = (torch.empty(n, d, device="cuda", dtype=torch.bfloat16).normal_(generator=g) for _ in range(2))
    w, rstd = torch.empty(d, device="cuda", dtype=torch.bfloat16).normal_(generator=g), torch.rand(n, device="cuda", generator=g)
    dx, dw = cp.rms_norm_grad(dy, x, rstd, w)
    part = 2**25
    dot = sum((dy[:, lo:lo + part].double() * w[lo:lo + part] * x[:, lo:lo + part]).sum(1) for lo in range(0, d, part))
    mean = (dot * rstd / d)[:, None]
    for lo in range(0, d, part):
        hat = x[:, lo:lo + part].double() * rstd[:, None]
        y = dy[:, lo:lo + part].double()
        want = (y * hat).sum(0)
        assert ((dw[lo:lo + part].double() - want).abs() <= (y * hat).abs().sum(0) * (n + 2) * 2.0**-24).all(), lo
        terms = (y * w[lo:lo + part]).abs() + (hat * mean).abs()
        want = rstd[:, None] * (y * w[lo:lo + part] - hat * mean)
        slack = want.abs() * 2.0**-8 + rstd[:, None] * terms * 8 * 2.0**-24 + rstd[:, None] * hat.abs() * 2.0**-20
        assert ((dx[:, lo:lo + part].double() - want).abs() <= slack).all(), lo


def test_norm_of_a_long_row():
    d = 2**28 + 3
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty(1, d, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    w = torch.empty(d, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    r = cp.rms_norm(x, w, rstd=True)
    part = 2**25
    mean = sum(x[0, lo:lo + part].double().square().sum() for lo in range(0, d, part)) / d
    root = torch.rsqrt(mean + 1e-6)
    assert abs(float(r.rstd) - float(root)) <= float(root) * 2.0**-10  # a sum of 2^18 terms a thread, in 32 bits
    for lo in range(0, d, part):
        want = x[0, lo:lo + part].double() * float(r.rstd) * w[lo:lo + part]
        assert ((r.y[0, lo:lo + part].double() - want).abs() <= want.abs() * 2.0**-8 + 1e-30).all(), lo
