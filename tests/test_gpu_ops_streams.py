"""The dense operators on a stream that is not torch's current one: what a call
allocates comes from that stream's memory, so that nothing it writes is still
in use by the current stream's work."""
from __future__ import annotations

import pytest
import torch

import trellis_coded_row_amd as cp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    torch.cuda.init()


def every_operator(inputs, stream):
    x, w, ids, table = inputs
    q = cp.quantize_fp8(x, transposed=True, stream=stream)
    r = cp.rms_norm(x, w, residual=x, fp8=True, rstd=True, stream=stream)
    product = cp.gemm_fp8(q[0][:100], q[1][:100], q[0][:70], q[1][:70], dtype=torch.float32, stream=stream)
    dx, dw = cp.rms_norm_grad(x, r.h, r.rstd, w, stream=stream)
    plan = cp.embed_plan(ids, table.shape[0], stream=stream)
    grad = cp.embed_grad(plan, x, stream=stream)
    rows = cp.embed_grad_rows(plan, x, stream=stream)
    out = cp.embed_lookup(table, ids, stream=stream)
    return [*q, r.h, r.y, r.q, r.scale, r.rstd, product, dx, dw, *plan[2:], grad, rows, out]


def inputs_of(n=6000, d=4992, rows=500):
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn(n, d, device="cuda", generator=g).bfloat16()
    return (x, torch.rand(d, device="cuda", generator=g).bfloat16(),
            torch.randint(0, rows, (n,), device="cuda", generator=g), torch.randn(rows, d, device="cuda", generator=g))


UNDEFINED_ENDS = (12, 13, 14, 15, 18)  # the plan's arrays and the distinct rows' gradient end before their tensors do


def bits(t):
    return t.contiguous().view(torch.uint8) if t.element_size() == 1 else t


@pytest.mark.parametrize("form", ["stream", "handle", "none", "zero"])
def test_allocations_are_the_streams_own(form):
    inputs = inputs_of()
    assert cp.cp_gemm_fp8_workspace_bytes(100, 70, 4992, cp.CP_DTYPE_F32) > 0  # workspaces are among them
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    given = {"stream": side, "handle": side.cuda_stream, "none": None, "zero": 0}[form]
    want = 0 if form in ("none", "zero") else side.cuda_stream
    torch.cuda.memory._record_memory_history(context=None)
    try:
        if form == "zero":  # the default stream, while another one is current
            with torch.cuda.stream(side):
                outs = every_operator(inputs, given)
                assert torch.cuda.current_stream() == side
        else:
            outs = every_operator(inputs, given)
            assert torch.cuda.current_stream() == torch.cuda.default_stream()
        made = [e for e in torch.cuda.memory._snapshot()["device_traces"][torch.cuda.current_device()]
                if e["action"] == "alloc"]
    finally:
        torch.cuda.memory._record_memory_history(enabled=None)
    torch.cuda.synchronize()
    assert len(made) >= 15 and {e["stream"] for e in made} == {want}
    for k, (a, b) in enumerate(zip(outs, every_operator(inputs, None))):
        if k not in UNDEFINED_ENDS:
            assert torch.equal(bits(a), bits(b)), k


def busy(x, rounds=40):
    """Work that keeps the current stream occupied for some milliseconds."""
    for _ in range(rounds):
        x = x @ x
    return x


def test_pending_work_on_the_current_stream_keeps_its_memory():
    n, d = 4096, 4096
    x, w = torch.randn(n, d, device="cuda").bfloat16(), torch.ones(d, device="cuda", dtype=torch.bfloat16)
    want = cp.rms_norm(x, w).y
    heavy = torch.randn(4096, 4096, device="cuda").bfloat16() * 0.01
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    temporary = torch.full((n, d), 3.0, device="cuda", dtype=torch.bfloat16)
    busy(heavy)
    read = temporary + 1  # waits for the work before it
    del temporary         # its memory is free to the current stream alone
    y = cp.rms_norm(x, w, stream=side).y
    torch.cuda.synchronize()
    assert (read == 4).all() and torch.equal(y, want)


def test_an_output_dropped_on_the_current_stream_stays_until_it_was_read():
    n, d = 4096, 4096
    x, w = torch.randn(n, d, device="cuda").bfloat16(), torch.ones(d, device="cuda", dtype=torch.bfloat16)
    want = cp.rms_norm(x, w).y
    heavy = torch.randn(4096, 4096, device="cuda").bfloat16() * 0.01
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = cp.rms_norm(x, w, stream=side).y
    torch.cuda.current_stream().wait_stream(side)
    busy(heavy)
    read = y + 0
    del y
    other = cp.rms_norm(x, w, residual=x, stream=side).y  # of the same size, on the side stream
    torch.cuda.synchronize()
    assert torch.equal(read, want + 0) and other.shape == want.shape


def test_a_branch_of_a_graph():
    inputs = inputs_of(n=3000, d=520)
    want = every_operator(inputs, None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        outs = every_operator(inputs, side)
        torch.cuda.current_stream().wait_stream(side)
    for r in range(3):
        for t in outs:
            t.view(torch.uint8).zero_() if t.element_size() == 1 else t.zero_()  # eager work between replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(outs, want)):
            if k not in UNDEFINED_ENDS:
                assert torch.equal(bits(a), bits(b)), f"replay {r}, output {k}"
    del graph
