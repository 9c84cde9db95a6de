"""The dense operators in a HIP graph and on other streams: every replay,
with eager work between, equals the eager result bit for bit."""
from __future__ import annotations

import pytest
import torch

import trellis_coded_row_amd as cp

pytestmark = pytest.mark.gpu
REPLAYS = 4


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    torch.cuda.init()


def steps(n, d, rows, hidden):
    """One training step of a row table and its readout, forward and back."""
    g = torch.Generator(device="cuda").manual_seed(n)
    table = torch.randn(rows, d, device="cuda", generator=g).bfloat16()
    ids = torch.randint(-1, rows, (n,), device="cuda", generator=g)
    w = torch.rand(d, device="cuda", generator=g).bfloat16()
    weight, ws, weight_t, ws_t = cp.quantize_fp8(torch.randn(hidden, d, device="cuda", generator=g), blocks=True,
                                                 transposed=True)
    dout = torch.randn(n, hidden, device="cuda", generator=g).bfloat16()

    def step():
        x = cp.embed_lookup(table, ids, scale=d**0.5)
        r = cp.rms_norm(x, w, fp8=True, rstd=True)
        y = cp.gemm_fp8(r.q, r.scale, weight, ws)
        q, s, qt, st = cp.quantize_fp8(dout, transposed=True)
        dy = cp.gemm_fp8(q, s, weight_t, ws_t)
        _, _, yt, yst = cp.quantize_fp8(r.y, transposed=True)
        dweight = cp.gemm_fp8(qt, st, yt, yst, dtype=torch.float32)
        dx, dw = cp.rms_norm_grad(dy, x, r.rstd, w)
        plan = cp.embed_plan(ids, rows)
        return [x, r.y, y, dy, dweight, dx, dw, cp.embed_grad(plan, dx, scale=d**0.5)]

    return step


@pytest.mark.parametrize("n,d,rows,hidden", [(48, 512, 1000, 256), (3000, 136, 5000, 200), (20_000, 512, 700, 512)])
def test_a_training_step_replayed_from_a_graph(n, d, rows, hidden):
    print(f"graph n={n} d={d} rows={rows} hidden={hidden}", flush=True)
    step = steps(n, d, rows, hidden)
    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for r in range(REPLAYS):
        for t in out:
            t.fill_(3.0)  # eager work between replays
        step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, (t, w) in enumerate(zip(out, want)):
            assert torch.equal(t, w), f"replay {r}, output {k}"
    del graph


def test_operators_on_a_stream_of_the_callers():
    step = steps(500, 64, 200, 128)
    want = step()
    torch.cuda.synchronize()
    x = torch.randn(2000, 700, device="cuda").bfloat16()
    ids = torch.randint(0, 300, (2000,), device="cuda")
    w = torch.ones(700, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    q = cp.quantize_fp8(x, transposed=True, stream=s)
    r = cp.rms_norm(x, w, fp8=True, rstd=True, stream=s)
    y = cp.gemm_fp8(q[0], q[1], q[0], q[1], stream=s)
    dx, dw = cp.rms_norm_grad(x, x, r.rstd, w, stream=s)
    plan = cp.embed_plan(ids, 300, stream=s)
    grad = cp.embed_grad(plan, x, stream=s)
    rows = cp.embed_lookup(grad, ids, stream=s)
    s.synchronize()
    q2 = cp.quantize_fp8(x, transposed=True)
    r2 = cp.rms_norm(x, w, fp8=True, rstd=True)
    assert torch.equal(q[0].view(torch.uint8), q2[0].view(torch.uint8)) and torch.equal(r.y, r2.y)
    assert torch.equal(y, cp.gemm_fp8(q2[0], q2[1], q2[0], q2[1]))
    dx2, dw2 = cp.rms_norm_grad(x, x, r2.rstd, w)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    grad2 = cp.embed_grad(cp.embed_plan(ids, 300), x)
    assert torch.equal(grad, grad2) and torch.equal(rows, cp.embed_lookup(grad2, ids))
    assert all(torch.equal(a, b) for a, b in zip(step(), want))
