"""What the dense operators' torch functions refuse before any launch."""
from __future__ import annotations

import pytest
import torch

import trellis_coded_row_amd as cp


def test_wrong_kinds_of_arguments():
    x, ids = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: cp.embed_lookup([1.0], ids), lambda: cp.embed_lookup(x, None),
                 lambda: cp.embed_plan(torch.tensor(3), 10), lambda: cp.embed_plan([1, 2], 10),
                 lambda: cp.rms_norm(None, x), lambda: cp.rms_norm_grad(x, x, None, None),
                 lambda: cp.quantize_fp8(3), lambda: cp.quantize_fp8(x.int()),
                 lambda: cp.gemm_fp8(x.to(torch.float8_e4m3fn), x, x, x),
                 lambda: cp.embed_grad(cp.EmbedPlan(4, 9, ids, ids, ids, ids, ids), x)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_wrong_tensors_on_the_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    x, ids = torch.zeros(4, 8, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    w = torch.ones(8, device="cuda")
    for call in (lambda: cp.embed_lookup(x, ids.int()), lambda: cp.embed_lookup(x.t(), ids), lambda: cp.embed_lookup(x, ids[::2]),
                 lambda: cp.embed_lookup(x, ids, dtype=torch.float64), lambda: cp.embed_lookup(x, ids, dtype="bf16"),
                 lambda: cp.embed_lookup(x, ids, out=x.half(), dtype=torch.float32), lambda: cp.embed_lookup(x, ids, out=x[:3]),
                 lambda: cp.embed_lookup(x, ids, bad_id=ids), lambda: cp.embed_lookup(x.int(), ids),
                 lambda: cp.embed_plan(ids, -1), lambda: cp.embed_grad(cp.embed_plan(ids, 5), x[:3]),
                 lambda: cp.rms_norm(x, w[:7]), lambda: cp.rms_norm(x, w.half()), lambda: cp.rms_norm(x, w, residual=x[:3]),
                 lambda: cp.rms_norm(x[:, :0], w[:0]), lambda: cp.rms_norm_grad(x.half(), x, ids.float(), w),
                 lambda: cp.rms_norm_grad(x, x, w, w)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: cp.embed_lookup(x, ids, scale="a"), lambda: cp.embed_plan(ids, 2.5),
                 lambda: cp.rms_norm(x, w, stream="s")):
        with pytest.raises((TypeError, ValueError)):
            call()
    with pytest.raises(cp.CPError):
        cp.embed_plan(ids, 2**62 + 1)
    # a handle, a stream and torch's current one give the same
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [cp.embed_lookup(x, ids, stream=s) for s in (None, side, side.cuda_stream, 0)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_the_gradient_of_too_long_rows_is_not_supported():
    p = 1 << 20  # a stand-in address, never dereferenced
    f = lambda d: cp.cp_embed_grad(p, p, p, p, p, 4, 10, p, cp.CP_DTYPE_F32, d, d, 1.0, p, p, 1 << 40, None)
    assert f(2**21 + 1) == cp.CP_ERR_UNSUPPORTED and f(2**31) == cp.CP_ERR_INVALID_ARGUMENT
    assert cp.cp_embed_grad_workspace_bytes(4, 2**21 + 1) == 0 and cp.cp_embed_grad_workspace_bytes(4, 2**21) > 0
