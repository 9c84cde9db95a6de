"""The 8-bit product's refusals at the far end of its sizes, without a GPU. The
calls run in a process of their own: what they must not do ends a process."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

import trellis_coded_row_amd as cp
from trellis_coded_row_amd import build as cpbuild

CALL = """
import trellis_coded_row_amd as cp
P = 1 << 20  # a stand-in address, never dereferenced: the call ends in its checks
m, n, code = {m}, {n}, {code}
print("status", cp.cp_gemm_fp8(P, 128, P, 4, P, 128, P, 4, 0, m, n, 128, P, n, code, None, 0, None))
"""


@pytest.mark.parametrize("m,n", [(2**25, 2**25), (2**25, 2**14), (2**16, 2**23), (2**25 - 255, 2**14 - 127)])
@pytest.mark.parametrize("code", [cp.CP_DTYPE_F32, cp.CP_DTYPE_BF16])
def test_more_tiles_than_a_launch_has(m, n, code):
    r = subprocess.run([sys.executable, "-c", CALL.format(m=m, n=n, code=code)], cwd=cpbuild.ROOT,
                       env=dict(os.environ, PYTHONPATH=cpbuild.ROOT), capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-400:]
    assert r.stdout.split() == ["status", str(cp.CP_ERR_UNSUPPORTED)]
    assert cp.cp_gemm_fp8_workspace_bytes(m, n, 128, code) == 0


def test_the_largest_products_have_a_workspace_size():
    # few rows by many columns and the reverse, one launch each: no splits of one step
    for m, n in ((64, 2**25), (2**25, 64), (2**25 - 256, 2**14 - 128), (2**16 - 256, 2**23)):
        for code in (cp.CP_DTYPE_F32, cp.CP_DTYPE_BF16):
            assert cp.cp_gemm_fp8_workspace_bytes(m, n, 128, code) == 0
    assert cp.cp_gemm_fp8_workspace_bytes(100, 64, 24576, cp.CP_DTYPE_F32) > 0
