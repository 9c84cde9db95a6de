"""The dense operators' torch functions refuse tensors whose values are in no
memory of their own (wrappers, transforms, lazy negatives) with an exception."""
from __future__ import annotations

import pytest
import torch

import trellis_coded_row_amd as cp


class Wrapper(torch.Tensor):
    """A tensor that calls itself one on the GPU and has no memory."""

    @staticmethod
    def __new__(cls, *shape, dtype=torch.float32):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device="cuda:0")

    @classmethod
    def __torch_dispatch__(cls, function, types, args=(), kwargs=None):
        raise NotImplementedError


def calls(x, ids, w, r, q, s, plan):
    return {"embed_lookup": lambda: cp.embed_lookup(x, ids, out=x, stream=0), "embed_plan": lambda: cp.embed_plan(ids, 9),
            "embed_grad": lambda: cp.embed_grad(cp.EmbedPlan(4, 9, *plan), x),
            "rms_norm": lambda: cp.rms_norm(x, w), "rms_norm_grad": lambda: cp.rms_norm_grad(x, x, r, w),
            "quantize_fp8": lambda: cp.quantize_fp8(x, stream=0), "gemm_fp8": lambda: cp.gemm_fp8(q, s, q, s, out=x)}


NAMES = ["embed_lookup", "embed_plan", "embed_grad", "rms_norm", "rms_norm_grad", "quantize_fp8", "gemm_fp8"]


@pytest.mark.parametrize("name", NAMES)
def test_tensors_without_memory(name):
    i32, i64 = torch.int32, torch.int64
    plan = [Wrapper(4, dtype=i32), Wrapper(4, dtype=i32), Wrapper(4, dtype=i64), Wrapper(5, dtype=i32), Wrapper(dtype=i64)]
    all_ = calls(Wrapper(4, 8), Wrapper(4, dtype=i64), Wrapper(8), Wrapper(4), Wrapper(4, 8, dtype=torch.float8_e4m3fn),
                 Wrapper(4, 1, dtype=torch.float8_e8m0fnu), plan)
    with pytest.raises(ValueError, match="memory of its own"):
        all_[name]()


def test_sparse_and_negated_host_tensors():
    ids, w = torch.zeros(4, dtype=torch.int64), torch.ones(8)
    for x in (torch.ones(4, 8).to_sparse(), torch._neg_view(torch.ones(4, 8))):
        for call in (lambda: cp.embed_lookup(x, ids), lambda: cp.rms_norm(x, w), lambda: cp.quantize_fp8(x)):
            with pytest.raises(ValueError, match="memory of its own"):
                call()


@pytest.mark.gpu
def test_transforms_on_the_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    x, w = torch.randn(3, 4, 8, device="cuda"), torch.ones(8, device="cuda")
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    out = torch.empty(4, 8, device="cuda")
    for function in (lambda t: cp.rms_norm(t, w).y, lambda t: cp.quantize_fp8(t)[0],
                     lambda t: cp.embed_lookup(t, ids, out=out), lambda t: cp.embed_lookup(x[0], ids, out=t)):
        with pytest.raises(ValueError, match="memory of its own"):
            torch.func.vmap(function)(x)
        with pytest.raises(ValueError, match="memory of its own"):
            torch.func.grad(lambda t: function(t).sum())(x[0])
    with pytest.raises(ValueError, match="memory of its own"):
        cp.rms_norm(torch._neg_view(x[0]), w)
    with torch._subclasses.FakeTensorMode(allow_non_fake_inputs=True) as mode:
        fake = mode.from_tensor(x[0])
        for call in (lambda: cp.rms_norm(fake, w), lambda: cp.quantize_fp8(fake), lambda: cp.embed_lookup(fake, ids, out=out)):
            with pytest.raises((ValueError, RuntimeError)):
                call()
    torch.cuda.synchronize()
    assert torch.equal(cp.embed_lookup(x[0], ids, out=out), x[0][ids])  # and goes on
