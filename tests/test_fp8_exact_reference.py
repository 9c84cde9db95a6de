"""The operands of the exact product tests tell an exact sum from the 8-bit
instruction's, shown with the instruction's cut-off in the oracle."""
from __future__ import annotations

import pytest
import torch

from fp8_exact_reference import cut_product, exponent, few_ones, packed, whole_numbers

SIZES = [(4, 9, 130), (3, 40, 4097), (2, 17, 24500), (2, 16, 24576)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_the_cut_off_shows_on_the_whole_numbers(m, n, k):
    x, y = whole_numbers(m, n, k, 1)
    exact = x.double() @ y.double().t()
    assert (x.abs().double() @ y.abs().double().t()).max() < 2**22
    assert (cut_product(x, y) != exact).double().mean() > 0.8
    # and so does one product left out, or counted twice
    at = int((x[0] != 0).nonzero()[k // 3 % int((x[0] != 0).sum())])
    for factor in (0.0, 2.0):
        z = x.clone()
        z[0, at] *= factor
        changed = (z.double() @ y.double().t())[0] != exact[0]
        assert torch.equal(changed, y[:, at] != 0) and changed.any()


@pytest.mark.parametrize("m,n,k", SIZES)
def test_the_few_ones_are_not_cut(m, n, k):
    x, y = few_ones(m, n, k, 2)
    exact = x.double() @ y.double().t()
    assert torch.equal(cut_product(x, y), exact) and exact.abs().max() <= 128
    x, y = whole_numbers(m, n, k, 3, large=False)
    assert torch.equal(cut_product(x, y), x.double() @ y.double().t())


def test_the_operands_are_in_e4m3_as_they_are():
    x, y = whole_numbers(5, 6, 200, 4)
    for t in (x, y):
        assert torch.equal(packed(t).float(), t) and packed(t).stride(0) == 208
    v = torch.tensor([0.0, 2.0**-9, 2.0**-6, 1.0, 1.875, 448.0])
    assert exponent(v).tolist() == [-6, -6, -6, 0, 0, 8]
