"""The smooth activations in the product's epilogue to their values' own size, also where they are far smaller than 1."""
from __future__ import annotations

import math

import pytest
import torch

import linear_reference as ref
import trellis_coded_row_amd as cp
from ops_reference import HALF

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]
# how far below 0 the exponential still is a normal number of 32 bits
DEPTH = {"silu": 85.0, "gelu": 13.0, "gelu_tanh": 9.5}
# z share(z) in units of 2^-24 of its size: an exponential 4 (the instruction's step is 2); 1 + e and its reciprocal 4.5, and two
# products 2; or gelu's polynomial, 3 for its argument, 3 for its sums, 2 for its coefficients, 1 for its fit, 1 for its
# product, and two more products and the difference from 1, 3: 17. Below the smallest normal exponential there may be 0.
# Where the result has 16 bits the exponent is one 32-bit number: its constant's, products' and sums' roundings count as often as
# it is large.
UNITS, LOST = 18, 2.0**-118


def exponent(z, name):
    """The roundings of the exponent of e, in units of 2^-24 of the power."""
    if name == "silu":
        return 1.25 * z.abs()
    return 1.1 * z * z if name == "gelu" else 4.5 * 2 * math.sqrt(2 / math.pi) * (z.abs() + 0.044715 * z.abs() ** 3)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    torch.cuda.init()


def places(name, dtype):
    gen = torch.Generator(device="cuda").manual_seed(4)
    low = DEPTH[name]
    whole = torch.arange(-int(low), 40, device="cuda").float()
    z = torch.cat([torch.linspace(-low, 0, 8000, device="cuda"), torch.randn(8000, device="cuda", generator=gen) * 3, whole,
                   torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e-6, -1e-6], device="cuda"), torch.linspace(0, 40, 2000, device="cuda")])
    return z.clamp(min=-low).to(dtype)


def check(got, z, name, what):
    dtype, z = got.dtype, z.double()
    want = ref.act(z, name)
    units = UNITS if dtype == torch.float32 else UNITS + exponent(z.clamp(max=0), name)
    off = units * ref.ULP * want.abs() + LOST * z.abs()
    off = off + HALF[dtype] * (want.abs() + off) + ref.TINY[dtype]
    ref.assert_near(got, want, off, f"{what} {name} {dtype}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
def test_values_to_their_own_size(name, dtype):
    z = places(name, dtype)
    empty = lambda m: torch.empty(m, 0, device="cuda", dtype=dtype)
    check(cp.linear(empty(1), empty(z.numel()), bias=z, act=name).y[0], z, name, "bias alone")
    one = lambda m: torch.eye(m, 64, device="cuda").to(dtype)
    for m in (1, 5, 64):  # four rows and sixteen at a time, and tiles
        w = z[: z.numel() // 64 * 64].view(-1, 64)
        for n in (w.shape[0], 40):
            check(cp.linear(one(m), w[:n], act=name).y, w[:n, :m].t(), name, f"{m} rows")


@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
def test_limits(name):
    """Infinities and values whose powers pass the largest number."""
    z = torch.tensor([math.inf, -math.inf, 3e38, -3e38, 1e13, -1e13, 9999.0, -9999.0, 10001.0, -10001.0, math.nan], device="cuda")
    y = cp.linear(torch.empty(1, 0, device="cuda"), torch.empty(11, 0, device="cuda"), bias=z, act=name).y[0].tolist()
    assert y[:10] == [v if v > 0 else 0 for v in z.tolist()[:10]] and math.isnan(y[10])
    dz, _ = cp.linear_act_grad(torch.ones(1, 11, device="cuda"), z.view(1, 11), act=name)
    dz = dz[0].tolist()
    assert dz[:10] == [1 if v > 0 else 0 for v in z.tolist()[:10]] and math.isnan(dz[10])
