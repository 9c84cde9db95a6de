"""The C entry points of include/cp_linear.h without a GPU: exported, bound, and refusing bad arguments on the host before
any HIP call."""
from __future__ import annotations

import ctypes
import math
import os
import re
import subprocess

import pytest

import trellis_coded_row_amd as cp
from trellis_coded_row_amd import build as cpbuild

HEADER = os.path.join(cpbuild.ROOT, "include", "cp_linear.h")
E, OK, U = cp.CP_ERR_INVALID_ARGUMENT, cp.CP_OK, cp.CP_ERR_UNSUPPORTED
F32, BF16, F16 = cp.CP_DTYPE_F32, cp.CP_DTYPE_BF16, cp.CP_DTYPE_F16
# stand-in addresses, never dereferenced: every call below ends in its checks
P, Q, R, S, T, V, W = (1 << k for k in (40, 41, 42, 43, 44, 45, 46))


def test_every_declared_symbol_is_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(cp_\w+)\s*\(", text)))
    assert len(names) == 9
    lib = ctypes.CDLL(cpbuild.LIB)
    for name in names:
        assert hasattr(lib, name) and callable(getattr(cp, name)), name
    from trellis_coded_row_amd import readout
    for name in readout.__all__:
        assert name in cp.__all__ and hasattr(cp, name)


def test_the_header_is_c_and_its_codes_are_the_bindings(tmp_path):
    src = tmp_path / "codes.c"
    src.write_text('#include <stdio.h>\n#include "cp_linear.h"\nint main(void) { printf("%d %d %d %d %d\\n", CP_ACT_NONE, '
                   'CP_ACT_RELU, CP_ACT_GELU, CP_ACT_GELU_TANH, CP_ACT_SILU); return 0; }\n')
    exe = tmp_path / "codes"
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in out] == [cp.CP_ACT_NONE, cp.CP_ACT_RELU, cp.CP_ACT_GELU, cp.CP_ACT_GELU_TANH, cp.CP_ACT_SILU]


def linear(x=P, xs=64, w=Q, ws=64, bias=R, res=S, rs=200, t=BF16, m=100, n=200, k=64, act=2, p=0.1, rng=T, y=V, ys=200, z=W,
           wsp=1 << 47, wb=1 << 40):
    return cp.cp_linear(x, xs, w, ws, bias, res, rs, t, m, n, k, act, p, rng, y, ys, z, wsp, wb, None)


def test_linear_checks():
    assert linear(t=3) == E and linear(t=-1) == E and linear(act=5) == E and linear(act=-1) == E
    for p in (-0.1, 1.0, 1.5, math.nan, math.inf, 1 - 2.0**-18):
        assert linear(p=p) == E, p
    assert linear(rng=None) == E and linear(rng=T + 4) == E
    for name in ("x", "w", "y"):
        assert linear(**{name: None}) == E, name
    for name, at in (("x", P), ("w", Q), ("bias", R), ("res", S), ("y", V), ("z", W)):
        assert linear(**{name: at + 1}) == E, name
        assert linear(t=F32, **{name: at + 2}) == E, name
    assert linear(ys=199) == E and linear(rs=2**61) == E
    assert linear(xs=2**22 + 1) == U and linear(ws=2**22 + 1) == U and linear(k=2**22 + 1, xs=2**22, ws=2**22) == U
    assert linear(m=2**25 + 1) == U and linear(n=2**25 + 1, ys=2**26, rs=2**26) == U
    assert linear(m=2**20, n=2**16, ys=2**16, rs=2**16) == U  # 2^24 tiles of 64 x 64
    assert linear(m=0) == OK and linear(n=0) == OK


def test_linear_workspaces():
    f = cp.cp_linear_workspace_bytes
    assert f(1, 512, 20000, BF16) > 0 and f(0, 5, 5, BF16) == f(5, 0, 5, F16) == f(5, 5, 0, F32) == 0
    assert f(5, 5, 5, 3) == 0 and f(2**26, 5, 5, BF16) == 0
    need = f(1, 512, 20000, BF16)
    call = lambda **a: linear(m=1, n=512, k=20000, xs=20000, ws=20000, ys=512, rs=512, **a)
    assert call(wb=need - 1) == E and call(wsp=None) == E and call(wsp=(1 << 47) + 128) == E
    assert cp.cp_linear_dx_workspace_bytes(100, 20000, 100, BF16) > 0 and cp.cp_linear_dw_workspace_bytes(20000, 100, 100, F16) > 0
    assert cp.cp_linear_dw_workspace_bytes(0, 100, 100, F16) == cp.cp_linear_dx_workspace_bytes(5, 0, 5, F32) == 0
    assert cp.cp_linear_act_grad_workspace_bytes(100, 100) > 0 and cp.cp_linear_act_grad_workspace_bytes(2**31, 1) == 0


def test_outputs_that_overlap_are_refused():
    size = 100 * 200 * 2
    assert linear(y=T) == E and linear(z=T) == E
    assert linear(y=P) == E and linear(y=Q + 64) == E and linear(y=R) == E and linear(z=V + size - 2) == E
    assert linear(z=P) == E and linear(z=S) == E and linear(res=V + 2) == E and linear(res=V, rs=201, ys=200) == E
    dx = lambda dz=P, w=Q, dres=None, out=V: cp.cp_linear_dx(dz, 200, w, 64, dres, 64, BF16, 100, 200, 64, out, 1 << 47, 1 << 40, None)
    assert dx(out=P) == E and dx(out=Q) == E and dx(dres=V + 2) == E
    dw = lambda dz=P, x=Q, out=V, add=0: cp.cp_linear_dw(dz, 200, x, 64, BF16, 100, 200, 64, add, out, 64, 1 << 47, 1 << 40, None)
    assert dw(out=P) == E and dw(out=Q + 4) == E and dw(out=V + 2) == E and dw(add=2) == E
    drop = lambda x=P, r=None, y=V, rng=T, p=0.5, xs=64: cp.cp_dropout(x, xs, r, 64, BF16, 100, 64, p, rng, y, None)
    assert drop(y=T) == E and drop(y=P + 2) == E and drop(y=P, xs=65) == E and drop(r=V + 4) == E
    grad = lambda dy=P, z=Q, dz=V, db=R, ds=64: cp.cp_linear_act_grad(dy, ds, z, 64, BF16, 100, 64, 4, 0.0, None, dz, db, 1 << 47,
                                                                    1 << 40, None)
    assert grad(dz=P + 2) == E and grad(dz=P, ds=70) == E and grad(dz=Q + 2) == E and grad(db=P) == E and grad(db=V) == E


def test_dx_and_dw_checks():
    dx = lambda dz=P, w=Q, dres=R, t=BF16, m=100, n=200, k=64, dx=V, ds=200, ws=64, rs=64, wsp=1 << 47, wb=1 << 40: \
        cp.cp_linear_dx(dz, ds, w, ws, dres, rs, t, m, n, k, dx, wsp, wb, None)
    assert dx(t=7) == E and dx(dz=None) == E and dx(w=None) == E and dx(dx=None) == E and dx(dres=R + 1) == E
    assert dx(ds=2**22 + 1) == U and dx(ws=2**22 + 1) == U and dx(n=2**22 + 1) == U and dx(m=2**25 + 1) == U
    assert dx(rs=2**61) == E and dx(m=0) == OK and dx(k=0) == OK
    assert dx(n=20000, k=100, wb=0) == E
    dw = lambda dz=P, x=Q, t=BF16, m=100, n=200, k=64, dw=V, ds=200, xs=64, os=64, wsp=1 << 47, wb=1 << 40: \
        cp.cp_linear_dw(dz, ds, x, xs, t, m, n, k, 0, dw, os, wsp, wb, None)
    assert dw(t=7) == E and dw(dz=None) == E and dw(x=None) == E and dw(dw=None) == E and dw(os=63) == E
    assert dw(ds=2**22 + 1) == U and dw(xs=2**22 + 1) == U and dw(m=2**25 + 1) == U and dw(n=2**22 + 1) == U
    assert dw(n=0) == OK and dw(k=0) == OK and dw(m=20000, n=100, k=100, os=100, wb=0) == E


def test_act_grad_and_dropout_checks():
    grad = lambda dy=P, z=Q, t=BF16, m=100, n=64, act=1, p=0.5, rng=T, dz=V, db=R, wsp=1 << 47, wb=1 << 40: \
        cp.cp_linear_act_grad(dy, 64, z, 64, t, m, n, act, p, rng, dz, db, wsp, wb, None)
    assert grad(t=9) == E and grad(act=6) == E and grad(p=1.0) == E and grad(rng=None) == E and grad(dy=None) == E
    assert grad(z=None) == E and grad(dz=None) == E and grad(db=R + 2) == E and grad(wb=0) == E and grad(wsp=None) == E
    assert grad(m=2**31) == E and grad(n=2**31) == E and grad(n=0) == OK and grad(m=0, db=None) == OK
    drop = lambda x=P, r=Q, t=BF16, n=100, d=64, p=0.5, rng=T, y=V: cp.cp_dropout(x, 64, r, 64, t, n, d, p, rng, y, None)
    assert drop(t=9) == E and drop(p=-1.0) == E and drop(p=math.nan) == E and drop(rng=None) == E and drop(x=None) == E
    assert drop(y=None) == E and drop(x=P + 1) == E and drop(r=Q + 1) == E and drop(n=2**31) == E and drop(d=2**31) == E
    assert drop(n=0) == OK and drop(d=0) == OK
