"""The 8-bit product where its exact result is known: 32-bit outputs of whole
numbers, equal to the last bit at any k (the 8-bit instruction's would not be:
test_fp8_exact_reference.py), 16-bit outputs where no product is cut, and the
cut itself, at the place that the header states."""
from __future__ import annotations

import pytest
import torch

import trellis_coded_row_amd as cp

from fp8_exact_reference import cut_product, few_ones, ones_scale, packed, whole_numbers
from ops_reference import groups

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]
# few rows (each kernel of them), and tiles of each size, with and without splits of k; ends inside steps and chunks
SIZES = [(1, 33, 24576), (16, 40, 4097), (17, 70, 24500), (33, 16, 24576), (64, 100, 4097), (100, 64, 24500),
         (200, 300, 4097), (513, 260, 24576), (700, 1030, 1153), (1500, 2100, 4097), (1030, 1024, 24500)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    torch.cuda.init()


def product(x, y, dtype, blocks=False):
    k = x.shape[1]
    scale = ones_scale(groups(y.shape[0]) if blocks else y.shape[0], k, "cuda")
    return cp.gemm_fp8(packed(x, "cuda"), ones_scale(x.shape[0], k, "cuda"), packed(y, "cuda"), scale, dtype=dtype)


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("blocks", [False, True])
def test_whole_numbers(m, n, k, blocks):
    print(f"whole numbers m={m} n={n} k={k} blocks={blocks}", flush=True)
    x, y = whole_numbers(m, n, k, m + n)
    assert torch.equal(product(x, y, torch.float32, blocks).double(), x.cuda().double() @ y.cuda().double().t())


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype", TYPES)
def test_every_product_counts_once(m, n, k, dtype):
    print(f"few ones m={m} n={n} k={k} {dtype}", flush=True)
    x, y = few_ones(m, n, k, m + n)
    assert torch.equal(product(x, y, dtype).double(), x.cuda().double() @ y.cuda().double().t())
    if dtype != torch.float32:  # sums of 22 bits, rounded once
        x, y = whole_numbers(m, n, k, m + n, large=False)
        assert torch.equal(product(x, y, dtype), (x.cuda().double() @ y.cuda().double().t()).to(dtype))


@pytest.mark.parametrize("m,n", [(16, 32), (48, 32), (130, 96), (600, 300), (4200, 4100)])
def test_where_a_16_bit_output_is_cut(m, n):
    # P - P + p with all three among 8 neighbouring k, or with p in other 8s: p is cut to a multiple of 2^-13 of P's
    # power of two in the first case and is summed in 32 bits in the second, as a 32-bit output's is in both: two sums
    # hold P, each off by at most 2^-23 of it
    k = 136
    print(f"cut m={m} n={n}", flush=True)
    g = torch.Generator().manual_seed(m)
    x, y = torch.zeros(m, k), torch.zeros(n, k)
    near = torch.arange(m) % 2 == 0
    first = 8 * torch.randint(0, k // 8 - 1, (m,), generator=g)
    rows = torch.arange(m)
    x[rows, first], x[rows, first + 1] = 256.0, -256.0
    x[rows, first + torch.where(near, 2, 8 + 5)] = torch.randint(1, 16, (m,), generator=g) / 8.0
    y[:] = 256.0
    y[:, 2::8] = y[:, 5::8] = torch.exp2(torch.randint(-6, 9, (n, 1), generator=g).float())
    want, cut = x.double() @ y.double().t(), cut_product(x[:200], y[:200])
    assert (cut != want[:200, :200])[near[:200]].any() and torch.equal(cut[~near[:200]], want[:200, :200][~near[:200]])
    off = 2 * 2.0**-23 * 2.0**16
    for dtype in (torch.bfloat16, torch.float16):
        out = product(x, y, dtype).double().cpu()[:200, :200]
        assert torch.equal(out[near[:200]], cut[near[:200]])  # multiples of 8
        assert ((out - cut).abs() <= off + cut.abs() * torch.finfo(dtype).eps / 2).all()
    assert ((product(x, y, torch.float32).double().cpu() - want).abs() <= off).all()
