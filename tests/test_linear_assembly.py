"""The products of the largest tile of the readout's product are written in assembly, whose latency the compiler does not
see: in the built kernels nothing but a product may touch an accumulator from the first product to the wait after the last
one, and nothing spills."""
from __future__ import annotations

import os
import re

import pytest

import test_gemm_assembly as gemm

KERNEL = "linear_tileILi%dELb%dELb%dELi%dELi4ELi4ELb%dE"
PRODUCT = r"v_mfma_f32_32x32x16_(?:bf16|f16) (a\[\d+:\d+\]), v\[\d+:\d+\], v\[\d+:\d+\], (a\[\d+:\d+\])"


@pytest.mark.skipif(not os.path.exists(os.path.join(gemm.LLVM, "llvm-objdump")), reason="no disassembler")
def test_the_accumulators_stay_in_place(tmp_path, monkeypatch):
    monkeypatch.setattr(gemm, "KERNEL", "linear_tileILi")
    found = {name: lines for name, lines in gemm.kernels(str(tmp_path)).items() if "ELi4ELi4ELb" in name}
    # two types, three layouts of the operands, whole chunks or rows at odd places
    wanted = [KERNEL % (t, a, b, out, direct) for t in (1, 2) for a, b, out in ((0, 0, t), (0, 1, t), (1, 1, 0)) for direct in (0, 1)]
    assert len(found) == len(wanted) == 12
    for part in wanted:
        (name, lines), = [(n, v) for n, v in found.items() if part in n]
        at = [i for i, line in enumerate(lines) if line.startswith("v_mfma")]
        # 64 products a step; five steps a turn and up to four after it, or two and one
        assert len(at) == 64 * (9 if part.endswith("1E") else 3), name
        for i in at:
            m = re.fullmatch(PRODUCT, lines[i])
            assert m and m.group(1) == m.group(2), f"{name}: {lines[i]}"
            assert lines[i - 1] == "s_nop 1", f"{name}: {lines[i - 1]}"
        uses = [i for i, line in enumerate(lines) if i not in set(at) and re.search(r"\ba(\d|\[)", line)]
        inside = [lines[i] for i in uses if at[0] < i < at[-1]]
        assert not inside, f"{name}: {inside[:3]}"
        assert not [line for line in lines if line.startswith("scratch_")], name
        after = min(i for i in uses if i > at[-1])
        waits = [i for i in range(at[-1], after) if lines[i] == "s_nop 15"]
        assert len(waits) >= 2, f"{name}: no wait before {lines[after]}"
