"""The dense operators' C entry points without a GPU: exported, bound, and
refusing bad arguments on the host before any HIP call."""
from __future__ import annotations

import ctypes
import os
import re

import pytest
import torch

import trellis_coded_row_amd as cp
from trellis_coded_row_amd import build as cpbuild

HEADER = os.path.join(cpbuild.ROOT, "include", "cp_ops.h")
E, OK, U = cp.CP_ERR_INVALID_ARGUMENT, cp.CP_OK, cp.CP_ERR_UNSUPPORTED
P = 1 << 20  # a stand-in address, never dereferenced: every call below ends in its checks
F32, BF16, F16 = cp.CP_DTYPE_F32, cp.CP_DTYPE_BF16, cp.CP_DTYPE_F16


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(cp_\w+)\s*\(", text)))


def test_every_declared_symbol_is_exported_and_bound():
    names = declared()
    assert len(names) == 11
    lib = ctypes.CDLL(cpbuild.LIB)
    for name in names:
        assert hasattr(lib, name), name
        assert callable(getattr(cp, name)), name
    for name in cp.ops.__all__:
        assert name in cp.__all__


def test_the_header_is_c_and_its_type_codes_are_the_bindings(tmp_path):
    import subprocess
    src = tmp_path / "codes.c"
    src.write_text('#include <stdio.h>\n#include "cp_ops.h"\n'
                   'int main(void) { printf("%d %d %d\\n", CP_DTYPE_F32, CP_DTYPE_BF16, CP_DTYPE_F16); return 0; }\n')
    exe = tmp_path / "codes"
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(cpbuild.ROOT, "include"), str(src), "-o",
                    str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in out] == [F32, BF16, F16]


def test_embed_lookup_checks():
    f = lambda table=P, tt=BF16, rows=10, d=8, stride=8, ids=P, n=4, out=P, ot=BF16, bad=None: \
        cp.cp_embed_lookup(table, tt, rows, d, stride, ids, n, 1.0, out, ot, bad, None)
    assert f(tt=3) == E and f(ot=-1) == E and f(ot=7) == E
    assert f(table=None) == E and f(table=P + 1) == E and f(ids=None) == E and f(ids=P + 4) == E
    assert f(out=None) == E and f(out=P + 1) == E and f(bad=P + 2) == E
    assert f(n=2**31) == E and f(d=2**31) == E and f(rows=2**62 + 1) == E
    assert f(rows=2**61, stride=2**40) == E
    assert f(n=0, ids=None, out=None) == OK and f(d=0, ids=None, out=None) == OK


def test_embed_plan_checks():
    need = cp.cp_embed_plan_workspace_bytes(100, 1000)
    assert need > 0 and cp.cp_embed_plan_workspace_bytes(0, 1000) == 0
    assert cp.cp_embed_plan_workspace_bytes(2**31, 1000) == 0
    f = lambda ids=P, n=100, rows=1000, order=P, slot=P, unique=P, starts=P, count=P, ws=P, wb=need: \
        cp.cp_embed_plan(ids, n, rows, order, slot, unique, starts, count, ws, wb, None)
    for k in ("ids", "order", "slot", "unique", "starts", "count", "ws"):
        assert f(**{k: None}) == E, k
    assert f(ids=P + 4) == E and f(order=P + 2) == E and f(unique=P + 4) == E and f(count=P + 4) == E
    assert f(ws=P + 64) == E and f(wb=need - 1) == E and f(n=2**31) == E and f(rows=2**63) == E
    assert f(n=0, starts=None) == E and f(n=0, count=None) == E


def test_embed_grad_checks():
    need = cp.cp_embed_grad_workspace_bytes(100, 64)
    f = lambda n=100, rows=0, dout=P, t=BF16, d=64, grad=P, ws=P, wb=need, order=P, starts=P, count=P: \
        cp.cp_embed_grad(order, P, P, starts, count, n, rows, dout, t, d, 64, 1.0, grad, ws, wb, None)
    assert f(t=3) == E and f(dout=None) == E and f(dout=P + 1) == E and f(grad=None) == E and f(order=None) == E
    assert f(starts=None) == E and f(count=P + 4) == E and f(ws=None) == E and f(wb=need - 1) == E
    assert f(n=2**31) == E and f(d=2**31) == E and f(rows=2**60, d=2**20) == E
    assert f(n=0) == OK and f(d=0) == OK


def test_rms_norm_checks():
    f = lambda x=P, res=None, w=P, t=BF16, n=4, d=130, h=None, y=P, q=None, qs=None, qst=144, sst=2, r=None: \
        cp.cp_rms_norm(x, 130, res, 130, w, t, n, d, 1e-6, h, y, q, qst, qs, sst, r, None)
    assert f(t=9) == E and f(d=0) == E and f(x=None) == E and f(x=P + 1) == E and f(w=None) == E
    assert f(h=P) == E                                  # no residual: h is x
    assert f(q=P) == E and f(qs=P) == E                 # both or neither
    assert f(q=P + 8, qs=P) == E and f(q=P, qs=P, qst=130) == E and f(q=P, qs=P, qst=128) == E
    assert f(q=P, qs=P, sst=1) == E and f(r=P + 2) == E and f(y=P + 1) == E and f(res=P + 1) == E
    assert f(n=2**31) == E and f(n=0) == OK


def test_rms_norm_grad_checks():
    need = cp.cp_rms_norm_grad_workspace_bytes(4, 64)
    f = lambda dy=P, x=P, r=P, w=P, dres=None, t=BF16, n=4, d=64, dx=P, dw=P, ws=P, wb=need: \
        cp.cp_rms_norm_grad(dy, 64, x, 64, r, w, dres, 64, t, n, d, dx, dw, ws, wb, None)
    for k in ("dy", "x", "r", "w", "dx", "ws"):
        assert f(**{k: None}) == E, k
    assert f(t=5) == E and f(d=0) == E and f(wb=need - 1) == E and f(dres=P + 1) == E and f(dw=P + 2) == E
    assert f(n=2**31) == E


def test_quantize_checks():
    f = lambda x=P, t=BF16, n=4, d=130, b=0, q=P, qst=144, s=P, sst=2, qt=None, qtst=16, st=None, stst=1: \
        cp.cp_quantize_fp8(x, t, n, d, 130, b, q, qst, s, sst, qt, qtst, st, stst, None)
    assert f(t=3) == E and f(b=2) == E and f(x=None) == E and f(q=None) == E and f(s=None) == E
    assert f(q=P + 8) == E and f(qst=130) == E and f(qst=128) == E and f(sst=1) == E
    assert f(qt=P) == E and f(st=P) == E and f(qt=P + 4, st=P) == E and f(qt=P, st=P, qtst=0) == E
    assert f(qt=P, st=P, stst=0) == E and f(n=2**31) == E
    assert f(n=0) == OK and f(d=0) == OK


def test_gemm_checks():
    assert cp.cp_gemm_fp8_workspace_bytes(4096, 4096, 4096, 5) == 0
    assert cp.cp_gemm_fp8_workspace_bytes(0, 10, 10, BF16) == 0
    f = lambda a=P, ast=144, sa=P, sast=4, b=P, bst=144, sb=P, sbst=4, blk=0, m=4, n=6, k=130, out=P, ost=6, t=BF16, \
        ws=None, wb=0: cp.cp_gemm_fp8(a, ast, sa, sast, b, bst, sb, sbst, blk, m, n, k, out, ost, t, ws, wb, None)
    assert f(t=3) == E and f(blk=2) == E
    for k in ("a", "b", "sa", "sb", "out"):
        assert f(**{k: None}) == E, k
    assert f(a=P + 8) == E and f(b=P + 1) == E and f(sa=P + 1) == E and f(sb=P + 2) == E and f(out=P + 1) == E
    assert f(ast=128) == E and f(ast=136) == E and f(bst=130) == E and f(sast=0) == E and f(sbst=2) == E
    assert f(ost=5) == E
    assert f(ast=2**23) == U and f(m=2**26) == U and f(n=2**26, ost=2**26) == U
    assert f(m=0) == OK and f(n=0) == OK
    need = cp.cp_gemm_fp8_workspace_bytes(100, 64, 24576, F32)
    if need:
        assert f(m=100, n=64, k=24576, ast=24576, bst=24576, sast=192, sbst=192, ost=64, t=F32, ws=P, wb=need - 1) == E


def test_the_torch_functions_refuse_host_tensors_and_wrong_types():
    x, w = torch.zeros(4, 8), torch.ones(8)
    ids = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: cp.embed_lookup(x, ids), lambda: cp.embed_plan(ids, 10), lambda: cp.rms_norm(x, w),
                 lambda: cp.rms_norm_grad(x, x, torch.ones(4), w), lambda: cp.quantize_fp8(x),
                 lambda: cp.gemm_fp8(x, x, x, x)):
        with pytest.raises(ValueError):
            call()
