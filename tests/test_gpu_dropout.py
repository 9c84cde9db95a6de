"""Dropout and the gradient through a product's epilogue, against the mask's definition and plain 64-bit forms."""
from __future__ import annotations

import pytest
import torch

import linear_reference as ref
import trellis_coded_row_amd as cp

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]
SIZES = [(1, 1), (1, 8), (3, 7), (5, 64), (1, 5000), (1000, 9), (33, 512), (129, 1030), (2000, 24), (70, 16400)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    torch.cuda.init()


def inputs(n, d, dtype):
    gen = torch.Generator(device="cuda").manual_seed(n * 31 + d)
    return (torch.randn(n, d, device="cuda", generator=gen).to(dtype), torch.randn(n, d, device="cuda", generator=gen).to(dtype),
            torch.randint(-(1 << 62), 1 << 62, (2,), device="cuda", generator=gen))


def expected(x, residual, p, rng):
    """One product and one sum in 32 bits, rounded once."""
    y = x.double()
    if p:
        mask, scale = ref.kept(rng.tolist(), p, *x.shape)
        y = torch.where(mask.cuda(), y * scale, torch.zeros_like(y))
    mag = y.abs()
    if residual is not None:
        y, mag = y + residual.double(), mag + residual.double().abs()
    return y, 4 * ref.ULP * mag + ref.rounding(y.abs() + 4 * ref.ULP * mag, x.dtype)


@pytest.mark.parametrize("n,d", SIZES)
@pytest.mark.parametrize("dtype", TYPES)
def test_dropout(n, d, dtype):
    print(f"dropout n={n} d={d} {dtype}", flush=True)
    x, residual, rng = inputs(n, d, dtype)
    for p in (0.0, 2.0**-16, 0.1, 0.5, 1 - 2.0**-16):
        for r in (None, residual):
            y = cp.dropout(x, p, rng, residual=r)
            ref.assert_near(y, *expected(x, r, p, rng), f"p {p}")
            if p:
                mask, _ = ref.kept(rng.tolist(), p, n, d)
                assert ((y == 0).cpu()[~mask]).all() if r is None else (y == r).cpu()[~mask].all()


@pytest.mark.parametrize("n,d", SIZES)
@pytest.mark.parametrize("dtype", TYPES)
def test_act_grad(n, d, dtype):
    print(f"act_grad m={n} n={d} {dtype}", flush=True)
    dy, z, rng = inputs(n, d, dtype)
    for name in ref.ACTS:
        for p in (0.0, 0.25):
            want, sums, off, off_db = ref.act_grad(dy, z, name, p, rng)
            dz, db = cp.linear_act_grad(dy, z if name else None, act=name, p=p, rng=rng)
            ref.assert_near(dz, want, off, f"dz {name}")
            ref.assert_near(db, sums, off_db, f"db {name}")
            other, none = cp.linear_act_grad(dy, z, act=name, p=p, rng=rng, db=False)
            assert none is None and torch.equal(other, dz)


def test_one_mask_everywhere():
    """The product's epilogue, its gradient and dropout drop the same places."""
    m, n = 150, 77
    _, _, rng = inputs(m, n, torch.float32)
    ones, eye = torch.ones(m, n, device="cuda"), torch.eye(m, device="cuda")
    alone = cp.dropout(ones, 0.4, rng)
    assert torch.equal(cp.linear(eye, ones.t().contiguous(), p=0.4, rng=rng).y, alone)
    assert torch.equal(cp.linear_act_grad(ones, p=0.4, rng=rng, db=False)[0], alone)
    mask, scale = ref.kept(rng.tolist(), 0.4, m, n)
    assert torch.equal(alone.cpu(), mask.float() * torch.tensor(scale).float())
    for k in range(2):
        other = rng.clone()
        other[k] += 1 << 33  # the high words count
        assert not torch.equal(cp.dropout(ones, 0.4, other), alone)


def test_the_share_that_is_dropped():
    """2^22 draws: within 5 deviations of sqrt(p (1 - p) / 2^22); rows, columns and offsets are not alike."""
    x = torch.ones(2048, 2048, device="cuda")
    for p in (0.1, 0.5, 0.9):
        for seed in range(3):
            rng = torch.tensor([seed, seed * 5], device="cuda")
            gone = (cp.dropout(x, p, rng) == 0).float()
            sigma = (p * (1 - p)) ** 0.5
            assert abs(float(gone.mean()) - p) < 5 * sigma / 2048
            for dim in (0, 1):
                assert ((gone.mean(dim) - p).abs() < 6 * sigma / 2048**0.5).all()
            moved = (cp.dropout(x, p, rng + 1) == 0).float()
            assert abs(float((gone * moved).mean()) - p * p) < 5 / 2048
            assert abs(float((gone[:, 1:] * gone[:, :-1]).mean()) - p * p) < 5 / 2048
            assert abs(float((gone[1:] * gone[:-1]).mean()) - p * p) < 5 / 2048


def test_what_is_dropped_is_zero_whatever_it_was():
    x = torch.full((40, 100), float("nan"), device="cuda")
    rng = torch.tensor([3, 4], device="cuda")
    y = cp.dropout(x, 0.5, rng)
    mask, _ = ref.kept([3, 4], 0.5, 40, 100)
    assert torch.isnan(y.cpu()[mask]).all() and (y.cpu()[~mask] == 0).all()
    dz, _ = cp.linear_act_grad(x, torch.full_like(x, float("inf")), act="gelu", p=0.5, rng=rng)
    assert torch.isnan(dz.cpu()[mask]).all() and (dz.cpu()[~mask] == 0).all()


def test_in_place_and_strides():
    for dtype in TYPES:
        x, residual, rng = inputs(300, 70, dtype)
        want = cp.dropout(x, 0.3, rng, residual=residual)
        a, b = x.clone(), residual.clone()
        assert cp.dropout(a, 0.3, rng, residual=residual, out=a) is a and torch.equal(a, want)
        assert cp.dropout(x, 0.3, rng, residual=b, out=b) is b and torch.equal(b, want)
        c = x.clone()
        assert torch.equal(cp.dropout(c, 0.3, rng, residual=c, out=c), cp.dropout(x, 0.3, rng, residual=x))
        wide = torch.full((301, 91), float("nan"), device="cuda", dtype=dtype)
        wide[:300, 5:75], part = x, wide[:300, 5:75]
        assert torch.equal(cp.dropout(part, 0.3, rng, residual=residual[:1].expand(300, 70)),
                           cp.dropout(x, 0.3, rng, residual=residual[:1].repeat(300, 1)))
        dz, db = cp.linear_act_grad(part, x[:1].expand(300, 70), act="silu", p=0.3, rng=rng)
        dz2, db2 = cp.linear_act_grad(x, x[:1].repeat(300, 1), act="silu", p=0.3, rng=rng)
        assert torch.equal(dz, dz2) and torch.equal(db, db2)
    assert cp.dropout(x[:0], 0.1, rng).shape == (0, 70) and cp.dropout(x[:, :0], 0.1, rng).shape == (300, 0)
