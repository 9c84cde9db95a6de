"""The dense operators on either side of a CP table (``include/cp_ops.h``).

Training the rows, before they are coded: ``embed_lookup`` reads an
uncompressed table, ``embed_plan`` groups a batch's ids by row and
``embed_grad`` / ``embed_grad_rows`` sum the lookup's gradient. The readout
of decoded rows: ``rms_norm`` and ``rms_norm_grad``, ``quantize_fp8`` and
``gemm_fp8``.

As in the rest of the package this module only marshals arguments; the
arithmetic runs in the library's HIP kernels. The functions named ``cp_*``
are the C entry points themselves (raw pointers and integers, a status
returned); the others take torch tensors on one GPU, allocate their outputs,
and raise ``ValueError`` for tensors they do not take and ``CPError`` for a
status other than CP_OK. ``stream=None`` is torch's current stream.

8-bit matrices are ``torch.float8_e4m3fn`` with ``torch.float8_e8m0fnu``
scales. Those made here have rows that start on 16 bytes (4 for scales), as
``gemm_fp8`` needs them.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import CP_OK, CPError, _L, _keep_for_stream, library_path

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

_CODE = {torch.float32: CP_DTYPE_F32, torch.bfloat16: CP_DTYPE_BF16, torch.float16: CP_DTYPE_F16}


def _bind(name: str, res, *args):
    if not hasattr(_L, name):
        raise ImportError(f"{library_path()} does not export {name}: it is older than its sources; "
                          "rebuild it (python trellis_coded_row_amd/build.py)")
    fn = getattr(_L, name)
    fn.restype = res
    fn.argtypes = args
    return fn


_vp, _u64, _int, _f32 = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_int, ctypes.c_float

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


# The calls for a single token's step end before their Python does, so what
# follows is kept short: torch.cuda.current_stream() makes an object (1.9 us
# of a call of 9 us), the two below return integers (0.07 and 0.14 us).
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _run(fn, device, stream, *args) -> None:
    """Calls a C entry point with `device` current, its stream last."""
    if stream is None:
        handle = _raw_stream(device.index)
    else:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if device.index == _current_device():
        st = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            st = fn(*args, handle)
    if st != CP_OK:
        raise CPError(st, fn.__name__)


def _matrix(t, name: str, dtype=None, shape=None) -> int:
    """Checks a 2-D device tensor whose rows are contiguous; its row stride."""
    if not t.is_cuda or t.dim() != 2 or (t.dtype not in _CODE if dtype is None else t.dtype != dtype):
        want = "float32, bfloat16 or float16" if dtype is None else dtype
        raise ValueError(f"{name} must be a 2-D {want} device tensor")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    stride, step = t.stride()
    if step != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return stride


def _vector(t, name: str, dtype, length: int, device) -> None:
    if not (t.is_cuda and t.dtype == dtype and t.shape == (length,) and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} device tensor of {length} values")
    _same(t, name, device)


def _same(t, name: str, device) -> None:
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")


def _ids(ids) -> int:
    if not (ids.is_cuda and ids.dtype == torch.int64 and ids.dim() == 1 and ids.is_contiguous()):
        raise ValueError("ids must be a contiguous 1-D int64 device tensor")
    return ids.shape[0]


def _fp8(rows: int, cols: int, device):
    """An empty rows x cols matrix of e4m3 whose rows start on 16 bytes."""
    if cols % 16 == 0:
        return torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device=device)
    return torch.empty((rows, cols + -cols % 16), dtype=torch.float8_e4m3fn, device=device)[:, :cols]


def _scales(rows: int, groups: int, device):
    """An empty rows x groups matrix of e8m0 whose rows start on 4 bytes."""
    if groups % 4 == 0:
        return torch.empty((rows, groups), dtype=torch.float8_e8m0fnu, device=device)
    return torch.empty((rows, groups + -groups % 4), dtype=torch.float8_e8m0fnu, device=device)[:, :groups]


def _workspace(nbytes: int, device, stream):
    """(tensor, pointer, bytes) of a call's scratch memory."""
    if nbytes == 0:
        return None, None, 0
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    _keep_for_stream(ws, stream)
    return ws, ws.data_ptr(), nbytes


# --------------------------------------------------------------------------
# embedding
# --------------------------------------------------------------------------

def embed_lookup(table, ids, scale: float = 1.0, dtype=None, out=None, bad_id=None, stream=None):
    """[n, d] of `dtype` (the table's, if None): scale * table[ids[j]], zeros
    for a negative id (padding) and for one past the table, which also sets
    `bad_id` (a device int32 tensor of one value) to 1 where given."""
    stride = _matrix(table, "table")
    n, (rows, d), device = _ids(ids), table.shape, table.device
    _same(ids, "ids", device)
    own = out is None
    if own:
        out = torch.empty((n, d), dtype=dtype or table.dtype, device=device)
        if stream is not None:
            _keep_for_stream(out, stream)
    elif not (out.is_cuda and out.dtype in _CODE and out.shape == (n, d) and out.is_contiguous()
              and dtype in (None, out.dtype)):
        raise ValueError(f"out must be a contiguous device tensor of shape ({n}, {d})")
    else:
        _same(out, "out", device)
    if out.dtype not in _CODE:
        raise ValueError("dtype must be float32, bfloat16 or float16")
    if bad_id is not None:
        _vector(bad_id, "bad_id", torch.int32, 1, device)
    _run(cp_embed_lookup, device, stream, table.data_ptr(), _CODE[table.dtype], rows, d, stride, ids.data_ptr(), n,
         scale, out.data_ptr(), _CODE[out.dtype], None if bad_id is None else bad_id.data_ptr())
    return out


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
    n, device = _ids(ids), ids.device
    if rows < 0:
        raise ValueError("rows must not be negative")
    order = torch.empty(n, dtype=torch.int32, device=device)
    slot = torch.empty(n, dtype=torch.int32, device=device)
    unique = torch.empty_like(ids)
    starts = torch.empty(n + 1, dtype=torch.int32, device=device)
    count = torch.empty((), dtype=torch.int64, device=device)
    ws, wp, wb = _workspace(cp_embed_plan_workspace_bytes(n, rows), device, stream)
    if stream is not None:
        for t in (order, slot, unique, starts, count):
            _keep_for_stream(t, stream)
    _run(cp_embed_plan, device, stream, ids.data_ptr(), n, rows, order.data_ptr(), slot.data_ptr(), unique.data_ptr(),
         starts.data_ptr(), count.data_ptr(), wp, wb)
    return EmbedPlan(n, rows, order, slot, unique, starts, count)


def _embed_grad(plan: EmbedPlan, dout, scale: float, whole: bool, stream):
    stride = _matrix(dout, "dout")
    n, d = dout.shape
    device = dout.device
    if n != plan.n:
        raise ValueError(f"dout has {n} rows, the plan {plan.n} lookups")
    _same(plan.order, "the plan", device)
    grad = torch.empty((plan.rows if whole else n, d), dtype=torch.float32, device=device)
    if grad.numel() == 0:
        return grad
    ws, wp, wb = _workspace(cp_embed_grad_workspace_bytes(n, d), device, stream)
    if stream is not None:
        _keep_for_stream(grad, stream)
    _run(cp_embed_grad, device, stream, plan.order.data_ptr(), plan.slot.data_ptr(), plan.unique.data_ptr(),
         plan.starts.data_ptr(), plan.count.data_ptr(), n, plan.rows if whole else 0, dout.data_ptr(),
         _CODE[dout.dtype], d, stride, scale, grad.data_ptr(), wp, wb)
    return grad


def embed_grad(plan: EmbedPlan, dout, scale: float = 1.0, stream=None):
    """float32 [rows, d]: the whole table's gradient of embed_lookup with the
    plan's ids, for the gradient dout [n, d] of its output."""
    return _embed_grad(plan, dout, scale, True, stream)


def embed_grad_rows(plan: EmbedPlan, dout, scale: float = 1.0, stream=None):
    """float32 [n, d]: row u < count is the gradient of table row
    plan.unique[u]; rows past plan.count are undefined."""
    return _embed_grad(plan, dout, scale, False, stream)


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
    xs = _matrix(x, "x")
    (n, d), device, dt = x.shape, x.device, x.dtype
    if d == 0:
        raise ValueError("x has no columns")
    _vector(weight, "weight", dt, d, device)
    h, rs = x, 0
    if residual is not None:
        rs = _matrix(residual, "residual", dt, x.shape)
        _same(residual, "residual", device)
        h = x.new_empty((n, d))
    out = x.new_empty((n, d)) if y else None
    q = sc = None
    if fp8:
        q, sc = _fp8(n, d, device), _scales(n, -(-d // FP8_GROUP), device)
    r = torch.empty(n, dtype=torch.float32, device=device) if rstd else None
    if stream is not None:
        for t in (h if residual is not None else None, out, q, sc, r):
            if t is not None:
                _keep_for_stream(t, stream)
    if n:
        _run(cp_rms_norm, device, stream, x.data_ptr(), xs, None if residual is None else residual.data_ptr(), rs,
             weight.data_ptr(), _CODE[dt], n, d, eps, None if residual is None else h.data_ptr(),
             out.data_ptr() if y else None, q.data_ptr() if fp8 else None, _row(q) if fp8 else 0,
             sc.data_ptr() if fp8 else None, _row(sc) if fp8 else 0, r.data_ptr() if rstd else None)
    return NormOut(h, out, q, sc, r)


def _row(t) -> int:
    """Bytes between the rows of a byte matrix."""
    return t.stride(0)


def rms_norm_grad(dy, x, rstd, weight, dres=None, stream=None):
    """(dx, dw) of rms_norm's y for its gradient dy: x is the norm's input
    (`h`, where there was a residual) and rstd what rms_norm kept. dx has x's
    type and includes dres, the gradient that reaches x past the norm, where
    given; dw is float32 [d]."""
    xs = _matrix(x, "x")
    (n, d), device, dt = x.shape, x.device, x.dtype
    if d == 0:
        raise ValueError("x has no columns")
    ys = _matrix(dy, "dy", dt, x.shape)
    _same(dy, "dy", device)
    _vector(rstd, "rstd", torch.float32, n, device)
    _vector(weight, "weight", dt, d, device)
    ds = 0
    if dres is not None:
        ds = _matrix(dres, "dres", dt, x.shape)
        _same(dres, "dres", device)
    dx = x.new_empty((n, d))
    dw = torch.empty(d, dtype=torch.float32, device=device)
    ws, wp, wb = _workspace(cp_rms_norm_grad_workspace_bytes(n, d), device, stream)
    if stream is not None:
        _keep_for_stream(dx, stream)
        _keep_for_stream(dw, stream)
    _run(cp_rms_norm_grad, device, stream, dy.data_ptr(), ys, x.data_ptr(), xs, rstd.data_ptr(), weight.data_ptr(),
         None if dres is None else dres.data_ptr(), ds, _CODE[dt], n, d, dx.data_ptr(), dw.data_ptr(), wp, wb)
    return dx, dw


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
    xs = _matrix(x, "x")
    (n, d), device = x.shape, x.device
    gn, gd = -(-n // FP8_GROUP), -(-d // FP8_GROUP)
    q, scale = _fp8(n, d, device), _scales(gn if blocks else n, gd, device)
    qt = scale_t = None
    if transposed:
        qt, scale_t = _fp8(d, n, device), _scales(gd if blocks else d, gn, device)
    if stream is not None:
        for t in (q, scale, qt, scale_t):
            if t is not None:
                _keep_for_stream(t, stream)
    if n and d:
        _run(cp_quantize_fp8, device, stream, x.data_ptr(), _CODE[x.dtype], n, d, xs, int(blocks), q.data_ptr(),
             _row(q), scale.data_ptr(), _row(scale), qt.data_ptr() if transposed else None,
             _row(qt) if transposed else 0, scale_t.data_ptr() if transposed else None,
             _row(scale_t) if transposed else 0)
    return q, scale, qt, scale_t


def _operand(t, name: str, dtype, unit: int, device):
    """Row stride of an 8-bit matrix whose rows start on `unit` bytes and can
    be read up to the next multiple of it."""
    stride = _matrix(t, name, dtype)
    _same(t, name, device)
    rows, cols = t.shape
    wide = -(-cols // unit) * unit
    if rows == 1:
        stride = wide
    if rows and cols:
        if stride % unit or stride < wide or t.data_ptr() % unit:
            raise ValueError(f"the rows of {name} must start on {unit} bytes")
        if wide != cols and t.untyped_storage().nbytes() < t.storage_offset() + (rows - 1) * stride + wide:
            raise ValueError(f"the last row of {name} must be readable up to a multiple of {unit} bytes")
    return stride if rows else wide


def gemm_fp8(a, a_scale, b, b_scale, dtype=torch.bfloat16, out=None, stream=None):
    """out [m, n] = A B^T of e4m3 matrices a [m, k] and b [n, k] with e8m0
    scales: a_scale [m, ceil(k / 128)], and b_scale either [n, ceil(k / 128)]
    or, one for each 128 x 128 block, [ceil(n / 128), ceil(k / 128)].
    Products are summed in 32 bits; dtype is float32, bfloat16 or float16."""
    device = a.device
    astride = _operand(a, "a", torch.float8_e4m3fn, 16, device)
    bstride = _operand(b, "b", torch.float8_e4m3fn, 16, device)
    sastride = _operand(a_scale, "a_scale", torch.float8_e8m0fnu, 4, device)
    sbstride = _operand(b_scale, "b_scale", torch.float8_e8m0fnu, 4, device)
    (m, k), n = a.shape, b.shape[0]
    groups = -(-k // FP8_GROUP)
    if b.shape[1] != k:
        raise ValueError(f"a has {k} columns, b {b.shape[1]}")
    if a_scale.shape != (m, groups):
        raise ValueError(f"a_scale must have shape ({m}, {groups})")
    if b_scale.shape == (n, groups):
        blocks = 0
    elif b_scale.shape == (-(-n // FP8_GROUP), groups):
        blocks = 1
    else:
        raise ValueError(f"b_scale must have shape ({n}, {groups}) or ({-(-n // FP8_GROUP)}, {groups})")
    if out is None:
        if dtype not in _CODE:
            raise ValueError("dtype must be float32, bfloat16 or float16")
        out = torch.empty((m, n), dtype=dtype, device=device)
        if stream is not None:
            _keep_for_stream(out, stream)
    else:
        if out.dtype != dtype:
            raise ValueError(f"out must have dtype {dtype}")
        ostride = _matrix(out, "out", None, torch.Size((m, n)))
        if m > 1 and ostride < n:
            raise ValueError("the rows of out must not overlap")
        _same(out, "out", device)
    ws, wp, wb = _workspace(cp_gemm_fp8_workspace_bytes(m, n, k, _CODE[out.dtype]), device, stream)
    _run(cp_gemm_fp8, device, stream, a.data_ptr(), astride, a_scale.data_ptr(), sastride, b.data_ptr(), bstride,
         b_scale.data_ptr(), sbstride, blocks, m, n, k, out.data_ptr(), out.stride(0) if m > 1 else n,
         _CODE[out.dtype], wp, wb)
    return out
