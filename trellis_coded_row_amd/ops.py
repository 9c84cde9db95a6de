"""The dense operators on either side of a CP table (``include/cp_ops.h``).

Training the rows, before they are coded: ``embed_lookup`` reads an
uncompressed table, ``embed_plan`` groups a batch's ids by row and
``embed_grad`` / ``embed_grad_rows`` sum the lookup's gradient. The readout
of decoded rows: ``rms_norm`` and ``rms_norm_grad``, ``quantize_fp8`` and
``gemm_fp8``.

As in the rest of the package the binding only marshals arguments; the
arithmetic runs in the library's HIP kernels. The functions named ``cp_*``
are the C entry points themselves (raw pointers and integers, a status
returned); the others take torch tensors on one GPU, allocate their outputs,
and raise ``ValueError`` for tensors they do not take and ``CPError`` for a
status other than CP_OK. Their checks, outputs and workspaces are made in C++
(``csrc/cp_torch.cpp``), as the calls of a single token's step take no longer
than their host side; where that library can be neither loaded nor built (no
compiler, for one), they raise ``ImportError`` and the rest of the package works.

``stream=None`` is torch's current stream. A call on another one (a stream or
its handle) does not wait for the current one: its inputs have to be ready
there and stay alive until it is done. What it allocates comes from that
stream's memory; an output may be dropped on the current stream after use there.

Nothing is recorded for autograd: the gradients are functions of their own, to
be called from a backward pass (an autograd function's forward and backward run
without recording). A tensor that requires a gradient is refused while torch
records, as its gradient would be lost.

8-bit matrices are ``torch.float8_e4m3fn`` with ``torch.float8_e8m0fnu``
scales. Those made here have rows that start on 16 bytes (4 for scales), as
``gemm_fp8`` needs them; a matrix and its scales share one allocation.
"""
from __future__ import annotations

import ctypes
import warnings
from typing import NamedTuple, Optional

import torch

from . import CPError, _L, library_path
from . import build as _build

__all__ = [
    "CP_DTYPE_F32", "CP_DTYPE_BF16", "CP_DTYPE_F16", "FP8_GROUP",
    "cp_embed_lookup", "cp_embed_plan_workspace_bytes", "cp_embed_plan", "cp_embed_grad_workspace_bytes",
    "cp_embed_grad", "cp_rms_norm", "cp_rms_norm_grad_workspace_bytes", "cp_rms_norm_grad", "cp_quantize_fp8",
    "cp_gemm_fp8_workspace_bytes", "cp_gemm_fp8",
    "EmbedPlan", "embed_lookup", "embed_plan", "embed_grad", "embed_grad_rows",
    "NormOut", "rms_norm", "rms_norm_grad", "quantize_fp8", "gemm_fp8",
]

CP_DTYPE_F32, CP_DTYPE_BF16, CP_DTYPE_F16 = 0, 1, 2
FP8_GROUP = 128  # values that share a scale


def _bind(name: str, res, *args):
    if not hasattr(_L, name):
        raise ImportError(f"{library_path()} does not export {name}: it is older than its sources; "
                          "rebuild it (python trellis_coded_row_amd/build.py)")
    fn = getattr(_L, name)
    fn.restype = res
    fn.argtypes = args
    return fn


_vp, _u64, _int, _f32, _f64 = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_int, ctypes.c_float, ctypes.c_double

cp_embed_lookup = _bind("cp_embed_lookup", _int, _vp, _int, _u64, _u64, _u64, _vp, _u64, _f32, _vp, _int, _vp, _vp)
cp_embed_plan_workspace_bytes = _bind("cp_embed_plan_workspace_bytes", _u64, _u64, _u64)
cp_embed_plan = _bind("cp_embed_plan", _int, _vp, _u64, _u64, _vp, _vp, _vp, _vp, _vp, _vp, _u64, _vp)
cp_embed_grad_workspace_bytes = _bind("cp_embed_grad_workspace_bytes", _u64, _u64, _u64)
cp_embed_grad = _bind("cp_embed_grad", _int, _vp, _vp, _vp, _vp, _vp, _u64, _u64, _vp, _int, _u64, _u64, _f32, _vp, _vp,
                      _u64, _vp)
cp_rms_norm = _bind("cp_rms_norm", _int, _vp, _u64, _vp, _u64, _vp, _int, _u64, _u64, _f32, _vp, _vp, _vp, _u64, _vp,
                    _u64, _vp, _vp)
cp_rms_norm_grad_workspace_bytes = _bind("cp_rms_norm_grad_workspace_bytes", _u64, _u64, _u64)
cp_rms_norm_grad = _bind("cp_rms_norm_grad", _int, _vp, _u64, _vp, _u64, _vp, _vp, _vp, _u64, _int, _u64, _u64, _vp, _vp,
                         _vp, _u64, _vp)
cp_quantize_fp8 = _bind("cp_quantize_fp8", _int, _vp, _int, _u64, _u64, _u64, _int, _vp, _u64, _vp, _u64, _vp, _u64, _vp,
                        _u64, _vp)
cp_gemm_fp8_workspace_bytes = _bind("cp_gemm_fp8_workspace_bytes", _u64, _u64, _u64, _u64, _int)
cp_gemm_fp8 = _bind("cp_gemm_fp8", _int, _vp, _u64, _vp, _u64, _vp, _u64, _vp, _u64, _int, _u64, _u64, _u64, _vp, _u64,
                    _int, _vp, _u64, _vp)


class _Unavailable:
    """In place of the C++ functions where they can be neither loaded nor
    built: the coded table does without them, a dense operator raises."""

    def __init__(self, reason: Exception):
        self.reason = reason

    def __getattr__(self, name):
        raise ImportError(f"{_build.TORCH_LIB}, which {name} runs on, can be neither loaded nor built: "
                          f"{type(self.reason).__name__}: {self.reason}") from self.reason


def _load_torch():
    """The functions of csrc/cp_torch.cpp; built first if they are not, or for
    another torch than the present one."""
    try:
        usable, present = _build.torch_built()
        if not usable:
            _build.build_torch()
        elif not present:
            warnings.warn(f"{_build.TORCH_LIB} is older than its sources; rebuild it "
                          "(python trellis_coded_row_amd/build.py)", stacklevel=2)
        from . import _cp_torch
        _cp_torch.setup(CPError)
    except Exception as e:
        return _Unavailable(e)
    return _cp_torch


_torch = _load_torch()


# --------------------------------------------------------------------------
# embedding
# --------------------------------------------------------------------------

def embed_lookup(table, ids, scale: float = 1.0, dtype=None, out=None, bad_id=None, stream=None):
    """[n, d] of `dtype` (the table's, if None): scale * table[ids[j]], zeros
    for a negative id (padding) and for one past the table, which also sets
    `bad_id` (a device int32 tensor of one value) to 1 where given."""
    return _torch.embed_lookup(table, ids, scale, dtype, out, bad_id, stream)


class EmbedPlan(NamedTuple):
    """A batch's ids grouped by row (cp_embed_plan): the lookups of row
    unique[u], for u < count, are order[starts[u]:starts[u + 1]], in batch
    order; slot[i] is the u of order[i], and -1 past them. Other entries past
    those are undefined."""
    n: int
    rows: int
    order: torch.Tensor   # int32[n]
    slot: torch.Tensor    # int32[n]
    unique: torch.Tensor  # int64[n], ascending
    starts: torch.Tensor  # int32[n + 1]
    count: torch.Tensor   # int64 scalar on the device


def embed_plan(ids, rows: int, stream=None) -> EmbedPlan:
    """Groups ids by row for embed_grad; ids outside [0, rows) take no part."""
    made = _torch.embed_plan(ids, rows, stream)
    return EmbedPlan(made[0].shape[0], rows, *made)


def embed_grad(plan: EmbedPlan, dout, scale: float = 1.0, stream=None):
    """float32 [rows, d]: the whole table's gradient of embed_lookup with the
    plan's ids, for the gradient dout [n, d] of its output."""
    return _torch.embed_grad(*plan, dout, scale, True, stream)


def embed_grad_rows(plan: EmbedPlan, dout, scale: float = 1.0, stream=None):
    """float32 [n, d]: row u < count is the gradient of table row
    plan.unique[u]; rows past plan.count are undefined."""
    return _torch.embed_grad(*plan, dout, scale, False, stream)


# --------------------------------------------------------------------------
# norm
# --------------------------------------------------------------------------

class NormOut(NamedTuple):
    """rms_norm's outputs; None where not asked for."""
    h: Optional[torch.Tensor]      # x + residual, x's type (x itself without a residual)
    y: Optional[torch.Tensor]      # the normed rows, x's type
    q: Optional[torch.Tensor]      # the normed rows in e4m3
    scale: Optional[torch.Tensor]  # e8m0, one for 128 values of a row
    rstd: Optional[torch.Tensor]   # float32 [n]


def rms_norm(x, weight, residual=None, eps: float = 1e-6, y: bool = True, fp8: bool = False, rstd: bool = False,
             stream=None) -> NormOut:
    """h = x + residual and y = h / sqrt(mean(h^2) + eps) * weight, row by
    row; y as a 16- or 32-bit matrix (`y`), in 8 bits (`fp8`), or both.
    `rstd` keeps 1 / sqrt(...) for rms_norm_grad."""
    return NormOut(*_torch.rms_norm(x, weight, residual, eps, y, fp8, rstd, stream))


def rms_norm_grad(dy, x, rstd, weight, dres=None, stream=None):
    """(dx, dw) of rms_norm's y for its gradient dy: x is the norm's input
    (`h`, where there was a residual) and rstd what rms_norm kept. dx has x's
    type and includes dres, the gradient that reaches x past the norm, where
    given; dw is float32 [d]."""
    return _torch.rms_norm_grad(dy, x, rstd, weight, dres, stream)


# --------------------------------------------------------------------------
# 8 bits
# --------------------------------------------------------------------------

def quantize_fp8(x, blocks: bool = False, transposed: bool = False, stream=None):
    """(q, scale, qt, scale_t) of a matrix x [n, d].

    q [n, d] in e4m3 with a scale for each 128 values of a row, scale
    [n, ceil(d / 128)]; with `blocks` one for each 128 x 128 block, scale
    [ceil(n / 128), ceil(d / 128)]. With `transposed`, qt [d, n] and scale_t
    are the same form of x transposed (with `blocks`: q and scale
    transposed); else None."""
    return _torch.quantize_fp8(x, blocks, transposed, stream)


def gemm_fp8(a, a_scale, b, b_scale, dtype=torch.bfloat16, out=None, stream=None):
    """out [m, n] = A B^T of e4m3 matrices a [m, k] and b [n, k] with e8m0
    scales: a_scale [m, ceil(k / 128)], and b_scale either [n, ceil(k / 128)]
    or, one for each 128 x 128 block, [ceil(n / 128), ceil(k / 128)].
    dtype is float32, bfloat16 or float16. Sums run in 32 bits; for the 16-bit
    types, of each 8 neighbouring products those far below the largest lose
    what lies 2^-13 below it (include/cp_ops.h), for float32 none does."""
    return _torch.gemm_fp8(a, a_scale, b, b_scale, dtype, out, stream)
