"""Parts of one wide matrix as inputs and outputs of a product: rows that lie between another's rows do not overlap them."""
from __future__ import annotations

import pytest
import torch

import trellis_coded_row_amd as cp

E, BF16 = cp.CP_ERR_INVALID_ARGUMENT, cp.CP_DTYPE_BF16
P, W, V = (1 << k for k in (40, 41, 44))  # stand-in addresses, never dereferenced: every call below ends in its checks


def test_rows_that_share_a_value_are_refused():
    """y has 64 of the 128 columns of a matrix of 100 rows."""
    def linear(x=W, xs=64, res=None, rs=0, bias=None, y=P, z=None, m=100, k=64):
        return cp.cp_linear(x, xs, W, 64, bias, res, rs, BF16, m, 64, k, 0, 0.0, None, y, 128, z, None, 0, None)
    for first in (-63, -1, 0, 1, 63, 65, 127):  # of x's columns, 64 too
        assert linear(x=P + 2 * first, xs=128) == E, first
        assert linear(x=P + 2 * (first + 128 * 7), xs=128) == E, first
    for first in (1, 63, 65, 127):
        assert linear(res=P + 2 * first, rs=128) == E
        assert linear(bias=P + 2 * (first + 128 * 3)) == E
    assert linear(x=P + 128, xs=127) == E and linear(x=P + 128, xs=129) == E  # not between them all the way
    assert linear(z=P + 128) == E and linear(x=P + 128, xs=128, k=65) == E
    dw = lambda x, xs: cp.cp_linear_dw(W, 64, x, xs, cp.CP_DTYPE_F32, 50, 40, 64, 0, V, 128, None, 0, None)
    assert dw(V + 4 * 63, 128) == E and dw(V + 4 * 65, 128) == E and dw(V + 4 * 64, 120) == E


@pytest.mark.gpu
def test_parts_of_one_matrix():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    stream = torch.cuda.current_stream().cuda_stream
    gen = torch.Generator(device="cuda").manual_seed(1)
    for m, n, k in ((1, 40, 64), (9, 64, 64), (130, 72, 100), (500, 64, 33)):
        wide = torch.randn(m, 2 * n + k + 8, device="cuda", generator=gen).bfloat16()
        before, w = wide.clone(), torch.randn(n, k, device="cuda", generator=gen).bfloat16()
        stride, at = wide.stride(0), lambda c: wide.data_ptr() + 2 * c
        need = cp.cp_linear_workspace_bytes(m, n, k, BF16)
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
        y, x, residual = wide[:, :n], wide[:, n:n + k], wide[:, n + k:2 * n + k]
        want = cp.linear(x.clone(), w, residual=residual.clone(), act="silu").y
        assert cp.cp_linear(at(n), stride, w.data_ptr(), k, None, at(n + k), stride, BF16, m, n, k, cp.CP_ACT_SILU, 0.0, None,
                            at(0), stride, None, ws.data_ptr(), need, stream) == cp.CP_OK
        assert torch.equal(y, want) and torch.equal(wide[:, n:], before[:, n:])
        # the bias in the first row's last columns
        assert n < 9 or cp.cp_linear(at(n), stride, w.data_ptr(), k, at(n + k), None, 0, BF16, m, n, k, cp.CP_ACT_NONE, 0.0, None,
                                     at(0), stride, None, ws.data_ptr(), need, stream) == cp.CP_OK
        assert torch.equal(y, cp.linear(x.clone(), w, bias=wide[0, n + k:2 * n + k].clone()).y)


@pytest.mark.gpu
def test_a_weights_gradient_beside_the_inputs():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    gen = torch.Generator(device="cuda").manual_seed(2)
    for n, k in ((40, 64), (130, 33)):
        wide = torch.randn(n, 2 * k, device="cuda", generator=gen)
        dz = torch.randn(n, n, device="cuda", generator=gen)
        x, into = wide[:, k:], wide[:, :k]
        want = cp.linear_dw(dz, x.clone(), into=into.clone())
        before = x.clone()
        assert torch.equal(cp.linear_dw(dz, x, into=into), want) and torch.equal(x, before)
