"""The dense operators record nothing for autograd: a tensor whose gradient
would be lost is refused, and under no_grad or in an autograd function the
calls and their gradients fit together."""
from __future__ import annotations

import pytest
import torch

import trellis_coded_row_amd as cp


def wanting(*shape, device="cpu"):
    return torch.ones(*shape, device=device, requires_grad=True)


def test_refused_while_torch_records():
    x, w, ids = wanting(4, 8), torch.ones(8), torch.zeros(4, dtype=torch.int64)
    plain, v = torch.ones(4, 8), wanting(8)
    plan = cp.EmbedPlan(4, 9, ids.int(), ids.int(), ids, torch.zeros(5, dtype=torch.int32), torch.tensor(1))
    calls = [lambda: cp.embed_lookup(x, ids), lambda: cp.embed_lookup(x + 1, ids), lambda: cp.embed_grad(plan, x),
             lambda: cp.embed_grad_rows(plan, x), lambda: cp.rms_norm(x, w), lambda: cp.rms_norm_grad(x, plain, w[:4], w),
             lambda: cp.quantize_fp8(x)]
    for call in calls:
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
        with torch.no_grad(), pytest.raises(ValueError) as refused:  # goes on to the next check: these are host tensors
            call()
        assert "gradient" not in str(refused.value)


@pytest.mark.gpu
def test_an_autograd_function_of_the_operators():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")

    class Readout(torch.autograd.Function):
        @staticmethod
        def forward(ctx, table, weight, ids):
            x = cp.embed_lookup(table, ids, scale=3.0)
            r = cp.rms_norm(x, weight, rstd=True)
            ctx.save_for_backward(x, r.rstd, weight, ids)
            ctx.rows = table.shape[0]
            return r.y

        @staticmethod
        def backward(ctx, dy):
            x, rstd, weight, ids = ctx.saved_tensors
            dx, dw = cp.rms_norm_grad(dy.contiguous(), x, rstd, weight)
            return cp.embed_grad(cp.embed_plan(ids, ctx.rows), dx, scale=3.0), dw, None

    g = torch.Generator(device="cuda").manual_seed(3)
    table = torch.randn(50, 40, device="cuda", generator=g, requires_grad=True)
    weight = torch.rand(40, device="cuda", generator=g, requires_grad=True)
    ids = torch.randint(0, 50, (200,), device="cuda", generator=g)
    dy = torch.randn(200, 40, device="cuda", generator=g)
    for call in (lambda: cp.embed_lookup(table, ids), lambda: cp.rms_norm(torch.ones(4, 40, device="cuda"), weight),
                 lambda: cp.rms_norm(torch.ones(4, 40, device="cuda"), weight.detach(), residual=table[:4]),
                 lambda: cp.embed_lookup(table.detach(), ids, out=wanting(200, 40, device="cuda"))):
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
    Readout.apply(table, weight, ids).backward(dy)
    t, w = (v.detach().double().cpu().requires_grad_() for v in (table, weight))
    x = t[ids.cpu()] * 3.0
    y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6) * w
    y.backward(dy.double().cpu())
    # 32-bit sums of up to 200 terms, each a few roundings off
    for got, want in ((table.grad, t.grad), (weight.grad, w.grad)):
        assert ((got.cpu().double() - want).abs() <= 256 * 2.0**-24 * (1 + want.abs().max())).all()
