"""The coded table's functions on a stream that is not torch's current one: what
a call allocates, and clears, is that stream's own."""
from __future__ import annotations

import pytest
import torch

import oracle
import trellis_coded_row_amd as cp
import workload

pytestmark = pytest.mark.gpu
ROWS, D, KV = 400, 64, 4


@pytest.fixture(scope="module")
def table():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    torch.cuda.init()
    lut = workload.lut_fp16(0)
    records, _ = oracle.encode_rows(workload.gaussian_rows(ROWS, D, seed=7), D, KV, lut, oracle.ENC_HEURISTIC)
    with cp.Table(ROWS, D, KV, lut) as t:
        t.upload(records)
        yield t


def every_function(table, ids, rows, stream):
    local, positions, counts = cp.shard_plan(ids, ROWS, 1, stream=stream)
    records = table.gather_records(ids, stream=stream)
    table.encode(rows, stream=stream)
    return [local, positions, counts, records, table.lookup_decode(ids, stream=stream),
            table.lookup_decode_raw(ids, stream=stream), table.lookup_decode_dedup(ids, stream=stream),
            table.lookup_decode_staged(records, ids.shape[0], positions, stream=stream)]


@pytest.mark.parametrize("form", ["stream", "handle", "zero", "none"])
def test_allocations_are_the_streams_own(table, form):
    ids = torch.randint(0, ROWS, (5000,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    rows = torch.randn(ROWS, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    side = torch.cuda.Stream()
    every_function(table, ids, rows, None)  # the table now holds the rows that each call encodes again
    want = every_function(table, ids, rows, None)
    torch.cuda.synchronize()
    given = {"stream": side, "handle": side.cuda_stream, "zero": 0, "none": None}[form]
    torch.cuda.memory._record_memory_history(context=None)
    try:
        if form == "zero":
            with torch.cuda.stream(side):
                outs = every_function(table, ids, rows, given)
        else:
            outs = every_function(table, ids, rows, given)
        made = [e for e in torch.cuda.memory._snapshot()["device_traces"][torch.cuda.current_device()]
                if e["action"] == "alloc"]
    finally:
        torch.cuda.memory._record_memory_history(enabled=None)
    torch.cuda.synchronize()
    assert len(made) >= 10
    assert {e["stream"] for e in made} == {side.cuda_stream if form in ("stream", "handle") else 0}
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    for k, (a, b) in enumerate(zip(outs, want)):
        assert torch.equal(a, b), k


def test_pending_work_on_the_current_stream_comes_in_no_way(table):
    # a buffer that was cleared on the current stream, behind its work, would be cleared after it was filled
    ids = torch.randint(0, ROWS, (20000,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    want, decoded = table.gather_records(ids), table.lookup_decode(ids)
    heavy = torch.randn(4096, 4096, device="cuda").bfloat16() * 0.01
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    temporary = torch.full((ids.shape[0], D), 3.0, device="cuda", dtype=torch.bfloat16)
    x = heavy
    for _ in range(40):
        x = x @ heavy
    read = temporary + 1
    del temporary
    records, out = table.gather_records(ids, stream=side), table.lookup_decode(ids, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(records, want) and torch.equal(out, decoded) and (read == 4).all()
