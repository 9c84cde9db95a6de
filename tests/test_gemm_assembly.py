"""The largest 8-bit tile's products are written in assembly, whose latency the
compiler does not see: in the built kernels nothing but a product may touch an
accumulator from the first product to the wait after the last one."""
from __future__ import annotations

import os
import re
import shutil
import subprocess

import pytest

from trellis_coded_row_amd import build as cpbuild

LLVM = "/opt/rocm/llvm/bin"
PRODUCT = "v_mfma_scale_f32_16x16x128_f8f6f4"
KERNEL = "gemm_tileILi8ELi8E"


def kernels(folder):
    """name -> instructions of the kernels with the largest tile in libcp.so."""
    lib = shutil.copy(cpbuild.LIB, folder)
    objdump = os.path.join(LLVM, "llvm-objdump")
    subprocess.run([objdump, "--offloading", lib], cwd=folder, check=True, capture_output=True)
    found = {}
    for name in sorted(os.listdir(folder)):
        if not name.endswith("gfx950"):
            continue
        with open(os.path.join(folder, name), "rb") as f:
            if KERNEL.encode() not in f.read():
                continue
        text = subprocess.run([objdump, "-d", "--no-show-raw-insn", name], cwd=folder, check=True, capture_output=True,
                              text=True).stdout
        lines = None
        for line in text.splitlines():
            head = re.match(r"^[0-9a-f]+ <(.*)>:$", line)
            if head:
                lines = found.setdefault(head.group(1), []) if KERNEL in head.group(1) else None
            elif lines is not None and line.startswith("\t"):
                lines.append(line.split("//")[0].strip())
    return found


@pytest.mark.skipif(not os.path.exists(os.path.join(LLVM, "llvm-objdump")), reason="no disassembler")
def test_the_accumulators_stay_in_place(tmp_path):
    found = kernels(str(tmp_path))
    assert len(found) == 4  # scales by block or row, k whole or with a tail
    for name, lines in found.items():
        at = [i for i, line in enumerate(lines) if line.startswith("v_mfma")]
        assert len(at) == 128, name  # 64 products, two steps a turn
        for i in at:
            m = re.fullmatch(PRODUCT + r" (a\[\d+:\d+\]), v\[\d+:\d+\], v\[\d+:\d+\], (a\[\d+:\d+\]), v\d+, v\d+ .*", lines[i])
            assert m and m.group(1) == m.group(2), f"{name}: {lines[i]}"
            assert lines[i - 1] == "s_nop 1", f"{name}: {lines[i - 1]}"
        uses = [i for i, line in enumerate(lines) if i not in set(at) and re.search(r"\ba(\d|\[)|scratch_", line)]
        inside = [lines[i] for i in uses if at[0] < i < at[-1]]
        assert not inside, f"{name}: {inside[:3]}"
        after = min(i for i in uses if i > at[-1])
        waits = [i for i in range(at[-1], after) if lines[i] == "s_nop 15"]
        assert len(waits) >= 2, f"{name}: no wait before {lines[after]}"
        back = [i for i in range(at[-1], waits[0]) if lines[i].startswith(("s_branch", "s_cbranch"))]
        assert back, name  # the loop ends before the wait
