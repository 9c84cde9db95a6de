"""A tensor that a dense operator writes into (out=, bad_id=) counts as changed
in place, so that autograd does not use it as a value saved before."""
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


def writers():
    table, ids = torch.randn(9, 32, device="cuda"), torch.arange(5, device="cuda")
    a, sa, _, _ = cp.quantize_fp8(torch.randn(5, 32, device="cuda"))
    b, sb, _, _ = cp.quantize_fp8(torch.randn(32, 32, device="cuda"))
    return (lambda out: cp.embed_lookup(table, ids, out=out),
            lambda out: cp.gemm_fp8(a, sa, b, sb, dtype=torch.float32, out=out))


def test_versions_count():
    for write in writers():
        out = torch.zeros(5, 32, device="cuda")
        for want in (1, 2):
            assert write(out) is out and out._version == want
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    made = cp.embed_lookup(torch.randn(9, 32, device="cuda"), torch.arange(12, device="cuda"), bad_id=bad)
    assert bad._version == 1 and int(bad) == 1 and made._version == 0
    with torch.inference_mode():
        out = torch.zeros(5, 32, device="cuda")
    for write in writers():
        write(out)  # has no version


def test_a_saved_value_that_was_written_over_is_noticed():
    for write in writers():
        x, out = torch.ones(5, 32, device="cuda", requires_grad=True), torch.ones(5, 32, device="cuda")
        y = x * out  # saves out
        write(out)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()
