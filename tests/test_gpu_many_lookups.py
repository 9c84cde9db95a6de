"""A lookup of more ids than one launch has waves for (2^30 and more), checked in
parts against small lookups of the same ids."""
from __future__ import annotations

import pytest
import torch

import oracle
import trellis_coded_row_amd as cp
import workload

pytestmark = pytest.mark.gpu
ROWS, D, KV = 512, 64, 4


@pytest.mark.parametrize("n", [2**30, 2**30 + 2**16 + 77])
def test_lookups_past_one_launch(n):
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    torch.cuda.empty_cache()
    need = n * (8 + 2 * D)
    if torch.cuda.mem_get_info()[0] < need + 2**35:
        pytest.skip("too little free memory")
    lut = workload.lut_fp16(0)
    records, _ = oracle.encode_rows(workload.gaussian_rows(ROWS, D, seed=5), D, KV, lut, oracle.ENC_HEURISTIC)
    ids = torch.empty(n, dtype=torch.int64, device="cuda")
    ids.random_(0, ROWS, generator=torch.Generator(device="cuda").manual_seed(1))
    out = torch.zeros(n, D, dtype=torch.bfloat16, device="cuda")
    with cp.Table(ROWS, D, KV, lut) as table:
        table.upload(records)
        rows = table.lookup_decode(torch.arange(ROWS, device="cuda"))
        table.lookup_decode(ids, out=out)
        assert table.check()
        part = 2**24
        for lo in range(0, n, part):
            assert torch.equal(out[lo:lo + part].view(torch.int16), rows[ids[lo:lo + part]].view(torch.int16)), lo
    del out, ids
    torch.cuda.empty_cache()
