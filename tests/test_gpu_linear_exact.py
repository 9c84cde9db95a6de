"""Products whose terms are 1 and -1, to the last bit: a term of K that is lost or counted twice changes a sum by 1 or 2,
which bounds by the sum of magnitudes need not show where K is long."""
from __future__ import annotations

import pytest
import torch

import trellis_coded_row_amd as cp

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]
# few rows: K whole, with a tail, in splits; tiles of each size, whole chunks and rows at odd places, splits, deep buffers
SIZES = [(1, 200, 4096), (1, 512, 20000), (3, 70, 20001), (4, 1000, 6000), (4, 5000, 300), (5, 33, 701), (8, 128, 24576),
         (16, 70, 1032), (16, 4100, 777), (17, 65, 130), (40, 100, 72), (64, 64, 24576), (65, 129, 201), (100, 1000, 40),
         (130, 72, 1000), (300, 520, 4100), (333, 7, 5001), (1030, 1000, 5000), (1000, 2050, 1030), (2048, 8192, 192),
         (2100, 2300, 1111), (4000, 4104, 328), (20000, 64, 33), (24576, 96, 104)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    torch.cuda.init()


def signs(gen, *shape):
    return torch.randint(0, 2, shape, device="cuda", generator=gen).float() * 2 - 1


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype", TYPES)
def test_whole_numbers(m, n, k, dtype):
    """Sums of up to 2^24 such terms are whole numbers that 32 bits hold; a result of 16 bits is one rounded once."""
    print(f"exact m={m} n={n} k={k} {dtype}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(m * 5 + n * 3 + k)
    x, w, dz = signs(gen, m, k), signs(gen, n, k), signs(gen, m, n)
    bias, residual, dres = (torch.randint(-9, 10, s, device="cuda", generator=gen).float() for s in ((n,), (m, n), (m, k)))
    t = [v.to(dtype) for v in (x, w, dz, bias, residual, dres)]
    wide = [v.double() for v in (x, w, dz, bias, residual, dres)]
    y = wide[0] @ wide[1].t()
    assert torch.equal(cp.linear(t[0], t[1]).y, y.float().to(dtype))
    got = cp.linear(t[0], t[1], bias=t[3], residual=t[4], act="relu", z=True)
    z = y + wide[3]
    assert torch.equal(got.z, z.float().to(dtype))
    assert torch.equal(got.y, (z.clamp(min=0) + wide[4]).float().to(dtype))
    dx = wide[2] @ wide[1]
    assert torch.equal(cp.linear_dx(t[2], t[1]), dx.float().to(dtype))
    assert torch.equal(cp.linear_dx(t[2], t[1], dres=t[5]), (dx + wide[5]).float().to(dtype))
    dw = (wide[2].t() @ wide[0]).float()
    assert torch.equal(cp.linear_dw(t[2], t[0]), dw)
    into = signs(gen, n, k)
    want = into + dw
    assert torch.equal(cp.linear_dw(t[2], t[0], into=into), want)


@pytest.mark.parametrize("m,n", [(1, 9), (3, 2050), (257, 64), (1000, 1030), (5000, 24), (70000, 130), (40, 16401), (300000, 8), (12000, 2056)])
@pytest.mark.parametrize("dtype", TYPES)
def test_sums_of_rows(m, n, dtype):
    """db of whole numbers, with relu's slopes of 0 and 1 and with half of them dropped (the others count twice)."""
    print(f"exact db m={m} n={n} {dtype}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(m + n)
    dy, z = signs(gen, m, n).to(dtype), signs(gen, m, n).to(dtype)
    dz, db = cp.linear_act_grad(dy)
    assert torch.equal(dz, dy) and torch.equal(db.double(), dy.double().sum(0))
    rng = torch.tensor([m, n], device="cuda")
    dz, db = cp.linear_act_grad(dy, z, act="relu", p=0.5, rng=rng)
    want = torch.where(z > 0, cp.dropout(dy, 0.5, rng), torch.zeros_like(dy))
    assert torch.equal(dz, want) and torch.equal(db.double(), want.double().sum(0))
