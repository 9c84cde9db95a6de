"""What the torch functions of the readout's product, its gradients and dropout refuse before any launch."""
from __future__ import annotations

import pytest
import torch

import trellis_coded_row_amd as cp
from test_ops_torch_wrappers import Wrapper


def test_wrong_kinds_of_arguments():
    x, w = torch.zeros(4, 8), torch.zeros(6, 8)
    for call in (lambda: cp.linear(None, w), lambda: cp.linear(x, [1.0]), lambda: cp.linear(x, w), lambda: cp.linear(x.int(), w),
                 lambda: cp.linear_act_grad(3), lambda: cp.linear_act_grad(x), lambda: cp.linear_dx(x, None),
                 lambda: cp.linear_dx(x, w), lambda: cp.linear_dw(x, 5), lambda: cp.linear_dw(x, x),
                 lambda: cp.dropout(None, 0.1, x), lambda: cp.dropout(x, 0.1, None)):
        with pytest.raises(ValueError):
            call()


def test_refused_while_torch_records():
    x, w = torch.ones(4, 8, requires_grad=True), torch.ones(6, 8)
    for call in (lambda: cp.linear(x, w), lambda: cp.linear(x.detach(), x), lambda: cp.linear_act_grad(x), lambda: cp.linear_dx(x, w),
                 lambda: cp.linear_dw(x, w), lambda: cp.dropout(x, 0.1, None)):
        with pytest.raises(ValueError, match="requires a gradient|device tensor"):
            call()


def test_tensors_without_memory():
    x, w, r = Wrapper(4, 8), Wrapper(6, 8), Wrapper(2, dtype=torch.int64)
    for call in (lambda: cp.linear(x, w), lambda: cp.linear_act_grad(x), lambda: cp.linear_dx(x, w), lambda: cp.linear_dw(x, x),
                 lambda: cp.dropout(x, 0.1, r)):
        with pytest.raises(ValueError, match="memory of its own"):
            call()


@pytest.mark.gpu
def test_wrong_tensors_on_the_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    x, w, y = torch.zeros(4, 8, device="cuda"), torch.zeros(6, 8, device="cuda"), torch.zeros(4, 6, device="cuda")
    rng = torch.zeros(2, dtype=torch.int64, device="cuda")
    into = torch.zeros(6, 8, device="cuda")
    bad = [lambda: cp.linear(x, w.half()), lambda: cp.linear(x, w[:, :7]), lambda: cp.linear(x[0], w), lambda: cp.linear(x.t(), w.t()),
           lambda: cp.linear(x.double(), w.double()), lambda: cp.linear(x, w, bias=x[0]), lambda: cp.linear(x, w, bias=y[0].half()),
           lambda: cp.linear(x, w, residual=x), lambda: cp.linear(x, w, residual=y.half()), lambda: cp.linear(x, w, act="tanh"),
           lambda: cp.linear(x, w, act=2), lambda: cp.linear(x, w, p=0.1), lambda: cp.linear(x, w, p=1.0, rng=rng),
           lambda: cp.linear(x, w, p=-0.1, rng=rng), lambda: cp.linear(x, w, p=float("nan"), rng=rng),
           lambda: cp.linear(x, w, p=0.1, rng=rng.int()), lambda: cp.linear(x, w, p=0.1, rng=rng[:1]),
           lambda: cp.linear(x, w, p=0.1, rng=rng.cpu()), lambda: cp.linear(x, w.cpu()),
           lambda: cp.linear_act_grad(y, act="relu"), lambda: cp.linear_act_grad(y, x, act="relu"),
           lambda: cp.linear_act_grad(y, y.half(), act="relu"), lambda: cp.linear_act_grad(y, p=0.5),
           lambda: cp.linear_dx(y, w.half()), lambda: cp.linear_dx(x, w), lambda: cp.linear_dx(y, w, dres=y),
           lambda: cp.linear_dw(y, x[:3]), lambda: cp.linear_dw(y, x.half()), lambda: cp.linear_dw(y, x, into=into.half()),
           lambda: cp.linear_dw(y, x, into=into[:5]), lambda: cp.linear_dw(y, x, into=into.t()),
           lambda: cp.linear_dw(y, x, into=into[:1].expand(6, 8)),
           lambda: cp.dropout(x, 0.1, None), lambda: cp.dropout(x, 2.0, rng), lambda: cp.dropout(x, 0.1, rng, residual=y),
           lambda: cp.dropout(x, 0.1, rng, out=y), lambda: cp.dropout(x, 0.1, rng, out=torch.zeros(4, 9, device="cuda")[:, :8])]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("taken:", k)
    for call in (lambda: cp.linear(x, w, p="a", rng=rng), lambda: cp.linear(x, w, stream="s"), lambda: cp.dropout(x, None, rng)):
        with pytest.raises((TypeError, ValueError)):
            call()
    flat = torch.zeros(200, device="cuda")
    for call in (lambda: cp.linear_dw(flat[:24].view(4, 6), flat[24:56].view(4, 8), into=flat[40:88].view(6, 8)),
                 lambda: cp.dropout(flat[:32].view(4, 8), 0.1, rng, out=flat[1:33].view(4, 8))):
        with pytest.raises(cp.CPError):  # an output that overlaps an input
            call()
    torch.cuda.synchronize()
