"""Slopes of the smooth activations to their own size, also where they are far smaller than 1."""
from __future__ import annotations

import math

import pytest
import torch

import linear_reference as ref
import trellis_coded_row_amd as cp
from ops_reference import HALF

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]
# how far below 0 the slope still is a normal number of 32 bits, with 32-bit exponentials on the way to it
DEPTH = {"silu": 85.0, "gelu": 13.0, "gelu_tanh": 9.5}
# A slope is share + z share', and its roundings count by the two terms' magnitudes, in units of 2^-24: the exponential 3 (the
# instruction's step is 2), 1 + e and its reciprocal 4.5, their product 1, and as much again for the second term's factor and its
# two products, 15 in all. A cubic through four such values has weights of at most 1.67 in sum: 25; its coefficients' roundings
# 10, its evaluation 4, and its own distance from the slope 5: 44. Below the smallest normal exponential there may be 0.
UNITS, LOST = 48, 2.0**-118


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    torch.cuda.init()


def terms(z, name):
    """The slope's two terms' magnitudes."""
    if name == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z.abs() * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    r = 2 * math.sqrt(2 / math.pi) if name == "gelu_tanh" else 1.0
    u = r * (z + 0.044715 * z**3) if name == "gelu_tanh" else z
    du = r * (1 + 3 * 0.044715 * z * z) if name == "gelu_tanh" else 1.0
    g = torch.sigmoid(u)
    return g + z.abs() * g * torch.sigmoid(-u) * du


def near(got, z, dy, scale, name, dtype):
    z, dy = z.double(), dy.double()
    want = ref.slope(z, name) * dy * scale
    # (the products with dy and the scale, and the scale's rounding)
    off = (UNITS * ref.ULP * terms(z, name) + LOST) * dy.abs() * scale + 3 * ref.ULP * want.abs()
    off = off + HALF[dtype] * (want.abs() + off) + ref.TINY[dtype]
    ref.assert_near(got, want, off, f"{name} {dtype}, z from {float(z.min())}")


def places(name, gen):
    """A tail, its neighbourhood, both sides of multiples of 1/64 and of whole numbers, values about 0."""
    low = DEPTH[name]
    grid = torch.arange(-640, 641, device="cuda") / 64
    whole = torch.arange(-int(low), 40, device="cuda").float()
    tiny = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e-6, -1e-6], device="cuda")
    up = lambda t, to: torch.nextafter(t, torch.full_like(t, to))
    z = torch.cat([torch.linspace(-low, 0, 30000, device="cuda"), torch.randn(30000, device="cuda", generator=gen) * 3, grid,
                   up(grid, 100.0), up(grid, -100.0), whole, up(whole, 100.0), up(whole, -100.0), tiny,
                   torch.linspace(0, 40, 5000, device="cuda")])
    return z.clamp(min=-low)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
def test_slopes_to_their_own_size(name, dtype):
    gen = torch.Generator(device="cuda").manual_seed(8)
    z = places(name, gen)
    n = 200
    z = z[: z.numel() // n * n].view(-1, n).to(dtype)
    dy = torch.randn(z.shape, device="cuda", generator=gen).to(dtype)
    for g in (torch.ones_like(z), dy):
        dz, _ = cp.linear_act_grad(g, z, act=name)
        near(dz, z, g, 1.0, name, dtype)
    rng = torch.tensor([3, 9], device="cuda")
    dz, _ = cp.linear_act_grad(dy, z, act=name, p=0.25, rng=rng)
    mask, scale = ref.kept([3, 9], 0.25, *z.shape)
    mask = mask.cuda()
    assert (dz[~mask] == 0).all()
    near(dz[mask], z[mask], dy[mask], scale, name, dtype)


@pytest.mark.parametrize("m,n", [(1, 9), (3, 1000), (4000, 520)])  # one row a thread, and several
@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
def test_all_of_a_batch_in_the_tail(name, m, n):
    gen = torch.Generator(device="cuda").manual_seed(m)
    z = -DEPTH[name] * torch.rand(m, n, device="cuda", generator=gen)
    dz, db = cp.linear_act_grad(torch.ones_like(z), z, act=name)
    near(dz, z, torch.ones_like(z), 1.0, name, torch.float32)
    want = ref.slope(z.double(), name).sum(0)
    off = (UNITS * ref.ULP * terms(z.double(), name) + LOST).sum(0) + (m + 2) * ref.ULP * ref.slope(z.double(), name).abs().sum(0)
    ref.assert_near(db, want, off + ref.TINY[torch.float32], "db")


@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
def test_a_deep_value_among_others_that_are_not(name):
    """One value of eight far below the others, in each place, and NaN and infinities beside it."""
    for low in (-5.5, -7.9, -8.1, -DEPTH[name]):
        z = torch.ones(64, 64, device="cuda")
        for i in range(64):
            z[i, i] = low
        z[0, 1], z[0, 2], z[0, 3] = float("nan"), float("inf"), -float("inf")
        z[1, 0] = -torch.tensor(float("nan"), device="cuda")
        dz, _ = cp.linear_act_grad(torch.ones_like(z), z, act=name)
        assert torch.isnan(dz[0, 1]) and torch.isnan(dz[1, 0]) and dz[0, 2] == 1 and dz[0, 3] == 0
        finite = torch.isfinite(z)
        near(dz[finite], z[finite], torch.ones_like(z)[finite], 1.0, name, torch.float32)
