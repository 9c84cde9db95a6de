"""NaN among the activation's inputs stays in its place of the gradient, and in its column of the sums."""
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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
def test_nan_stays_in_its_place(name, dtype):
    gen = torch.Generator(device="cuda").manual_seed(3)
    for m, n in ((1, 1), (7, 64), (70, 1030), (5000, 24)):
        z = (torch.randn(m, n, device="cuda", generator=gen) * 4).to(dtype)
        at = torch.rand(m, n, device="cuda", generator=gen) < 2 / m
        at[0, 0] = True
        bits = torch.int32 if dtype == torch.float32 else torch.int16
        one = torch.full_like(z, float("nan")).view(bits) | torch.randint(0, 1 << 7, (m, n), device="cuda", generator=gen).to(bits)
        sign = torch.where(torch.rand(m, n, device="cuda", generator=gen) < 0.5, torch.iinfo(bits).min, 0).to(bits)
        dirty = torch.where(at, (one | sign).view(dtype), z)
        assert torch.equal(torch.isnan(dirty), at)
        dy = torch.ones_like(z)
        want, _ = cp.linear_act_grad(dy, z, act=name)
        dz, db = cp.linear_act_grad(dy, dirty, act=name)
        assert torch.equal(torch.isnan(dz), at) and torch.equal(dz[~at], want[~at])
        assert torch.equal(torch.isnan(db), at.any(0))
