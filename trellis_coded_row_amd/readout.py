"""The readout's product in 16 and 32 bits, its gradients, and dropout (``include/cp_linear.h``).

``linear`` is a product with a bias, an activation, dropout and a residual in
its epilogue; ``linear_act_grad`` goes back through that epilogue, and
``linear_dx`` and ``linear_dw`` are the two products of the backward pass.
``dropout`` is the mask on its own. A layer's step, forward and back::

    r = linear(x, weight, bias, residual=h, act="gelu", p=0.1, rng=rng, z=True)   # r.y
    dz, db = linear_act_grad(dy, r.z, act="gelu", p=0.1, rng=rng)
    dx = linear_dx(dz, weight)
    dw = linear_dw(dz, x)                                 # the residual's gradient is dy

``rng`` is a device tensor of two int64 numbers, seed and offset, from which
the mask follows; none is stored. The gradient needs the same two numbers as
the forward pass, two masks two different offsets. They are read when the
kernel runs, so a captured graph that adds to the offset has another mask at
each replay.

As the functions of ``ops``: torch tensors on one GPU, ``ValueError`` for
tensors they do not take and ``CPError`` for a status other than CP_OK,
``stream`` as there, nothing recorded for autograd. The ``cp_*`` names are the
C entry points themselves.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from .ops import _bind, _f64, _int, _torch, _u64, _vp

__all__ = [
    "CP_ACT_NONE", "CP_ACT_RELU", "CP_ACT_GELU", "CP_ACT_GELU_TANH", "CP_ACT_SILU",
    "cp_linear_workspace_bytes", "cp_linear", "cp_linear_act_grad_workspace_bytes", "cp_linear_act_grad",
    "cp_linear_dx_workspace_bytes", "cp_linear_dx", "cp_linear_dw_workspace_bytes", "cp_linear_dw", "cp_dropout",
    "LinearOut", "linear", "linear_act_grad", "linear_dx", "linear_dw", "dropout",
]

CP_ACT_NONE, CP_ACT_RELU, CP_ACT_GELU, CP_ACT_GELU_TANH, CP_ACT_SILU = 0, 1, 2, 3, 4

cp_linear_workspace_bytes = _bind("cp_linear_workspace_bytes", _u64, _u64, _u64, _u64, _int)
cp_linear = _bind("cp_linear", _int, _vp, _u64, _vp, _u64, _vp, _vp, _u64, _int, _u64, _u64, _u64, _int, _f64, _vp, _vp,
                  _u64, _vp, _vp, _u64, _vp)
cp_linear_act_grad_workspace_bytes = _bind("cp_linear_act_grad_workspace_bytes", _u64, _u64, _u64)
cp_linear_act_grad = _bind("cp_linear_act_grad", _int, _vp, _u64, _vp, _u64, _int, _u64, _u64, _int, _f64, _vp, _vp, _vp,
                           _vp, _u64, _vp)
cp_linear_dx_workspace_bytes = _bind("cp_linear_dx_workspace_bytes", _u64, _u64, _u64, _u64, _int)
cp_linear_dx = _bind("cp_linear_dx", _int, _vp, _u64, _vp, _u64, _vp, _u64, _int, _u64, _u64, _u64, _vp, _vp, _u64, _vp)
cp_linear_dw_workspace_bytes = _bind("cp_linear_dw_workspace_bytes", _u64, _u64, _u64, _u64, _int)
cp_linear_dw = _bind("cp_linear_dw", _int, _vp, _u64, _vp, _u64, _int, _u64, _u64, _u64, _int, _vp, _u64, _vp, _u64, _vp)
cp_dropout = _bind("cp_dropout", _int, _vp, _u64, _vp, _u64, _int, _u64, _u64, _f64, _vp, _vp, _vp)


class LinearOut(NamedTuple):
    """linear's outputs; z is None where not asked for."""
    y: torch.Tensor            # [m, n], x's type
    z: Optional[torch.Tensor]  # the activation's input, rounded to x's type


def linear(x, weight, bias=None, residual=None, act: Optional[str] = None, p: float = 0.0, rng=None, z: bool = False,
           stream=None) -> LinearOut:
    """y = drop(act(x weight^T + bias)) + residual for x [m, k] and weight
    [n, k] of one type (float32, bfloat16 or float16), bias [n] and residual
    [m, n] of the same. act is None, "relu", "gelu", "gelu_tanh" or "silu"; p is
    the share that is dropped (0: none, rng is not read). `z` keeps the
    activation's input for linear_act_grad."""
    return LinearOut(*_torch.linear(x, weight, bias, residual, act, p, rng, z, stream))


def linear_act_grad(dy, z=None, act: Optional[str] = None, p: float = 0.0, rng=None, db: bool = True, stream=None):
    """(dz, db) for linear's gradient dy [m, n]: dz = drop(dy) act'(z), of dy's
    type, and db, float32 [n], the bias's gradient (None without `db`). z is what
    linear kept (not read without an activation); act, p and rng are linear's."""
    return _torch.linear_act_grad(dy, z, act, p, rng, db, stream)


def linear_dx(dz, weight, dres=None, stream=None):
    """dx [m, k] = dz weight, of dz's type, with dres added, the gradient that
    reaches x past the product, where given."""
    return _torch.linear_dx(dz, weight, dres, stream)


def linear_dw(dz, x, into=None, stream=None):
    """dw [n, k] = dz^T x in float32; added to `into`, in place, where that is
    given (which is then returned)."""
    return _torch.linear_dw(dz, x, into, stream)


def dropout(x, p: float, rng, residual=None, out=None, stream=None):
    """x [n, d] with the share p dropped and the rest divided by 1 - p, plus
    residual where given; into `out` (contiguous; x or residual themselves, for
    one), or a new tensor. The gradient is dropout(dy, p, rng)."""
    return _torch.dropout(x, p, rng, residual, out, stream)
