"""The readout's product, its gradients and dropout as a program uses them together: a layer's training step against 64
bits and against differences, replays from a graph, other streams, tensors that are written in place."""
from __future__ import annotations

import pytest
import torch

import linear_reference as ref
import trellis_coded_row_amd as cp

pytestmark = pytest.mark.gpu
REPLAYS = 4


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    torch.cuda.init()


class Layer(torch.autograd.Function):
    """linear with its gradients, and the residual's."""

    @staticmethod
    def forward(ctx, x, w, b, residual, rng, act, p):
        r = cp.linear(x, w, b, residual, act, p, rng, z=True)
        ctx.save_for_backward(x, w, r.z, rng)
        ctx.how = act, p
        return r.y

    @staticmethod
    def backward(ctx, dy):
        x, w, z, rng = ctx.saved_tensors
        act, p = ctx.how
        dy = dy.contiguous()
        dz, db = cp.linear_act_grad(dy, z, act, p, rng)
        return cp.linear_dx(dz, w), cp.linear_dw(dz, x).to(w.dtype), db.to(w.dtype), dy, None, None, None


class Drop(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, p, rng):
        ctx.save_for_backward(rng)
        ctx.p = p
        return cp.dropout(x, p, rng)

    @staticmethod
    def backward(ctx, dy):
        return cp.dropout(dy.contiguous(), ctx.p, ctx.saved_tensors[0]), None, None


def network(tokens, slots, d, hidden, gen):
    """Looked-up rows through dropout, a wide layer and one back to the residual stream."""
    width = slots * d
    normal = lambda *s, scale=1.0: torch.randn(*s, device="cuda", generator=gen) * scale
    parameters = [normal(tokens, width), normal(hidden, width, scale=width**-0.5), normal(hidden, scale=0.1),
                  normal(d, hidden, scale=hidden**-0.5), normal(d, scale=0.1), normal(tokens, d)]
    rngs = [torch.tensor([77, k], device="cuda") for k in range(3)]
    return [t.requires_grad_() for t in parameters], rngs


def forward(t, rngs, act, p):
    x, w1, b1, w2, b2, stream = t
    h = Layer.apply(Drop.apply(x, p, rngs[0]), w1, b1, torch.zeros(x.shape[0], w1.shape[0], device=x.device), rngs[1], act, p)
    return Layer.apply(h, w2, b2, stream, rngs[2], None, p)


def plain(t, rngs, act, p):
    """The same in 64 bits, by torch's own recording."""
    def drop(v, rng):
        if not p:
            return v
        mask, scale = ref.kept(rng.tolist(), p, *v.shape)
        return v * mask.to(v.device) * scale
    x, w1, b1, w2, b2, stream = t
    h = drop(ref.act(drop(x, rngs[0]) @ w1.t() + b1, act), rngs[1])
    return drop(h @ w2.t() + b2, rngs[2]) + stream


@pytest.mark.parametrize("act", ref.ACTS)
def test_a_layer_stack_and_its_gradients(act):
    """32-bit sums of up to 300 terms through two layers: a few hundred steps of 2^-24 of the values' size."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    for tokens, slots, d, hidden, p in ((70, 4, 30, 100, 0.2), (33, 3, 64, 128, 0.0), (1, 5, 16, 40, 0.5)):
        t, rngs = network(tokens, slots, d, hidden, gen)
        dy = torch.randn(tokens, d, device="cuda", generator=gen)
        y = forward(t, rngs, act, p)
        y.backward(dy)
        wide = [v.detach().double().requires_grad_() for v in t]
        want = plain(wide, rngs, act, p)
        want.backward(dy.double())
        for got, exact in [(y, want)] + [(a.grad, b.grad) for a, b in zip(t, wide)]:
            assert ((got.double() - exact).abs() <= 512 * ref.ULP * (exact.abs() + exact.abs().max())).all()


@pytest.mark.parametrize("act", ref.ACTS)
def test_gradients_against_differences(act):
    """Along random directions v: (f(t + h v) - f(t - h v)) / 2h of the function in 64 bits against the gradient's product
    with v. The gradient's values are within 512 steps of 2^-24 of their own size and the largest's (the test above), which
    the product with v sums up. With h = 2^-20 the difference is off by h^2 times a third derivative, 2^-40 of the values'
    size to the third power at most, and by 2^-52 / h of f's terms. relu's difference is off where a value crosses 0 on the
    way: by at most half of the slope's jump, 1, times that value's own change and gradient."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    t, rngs = network(64, 2, 40, 96, gen)
    dy = torch.randn(64, 40, device="cuda", generator=gen)
    forward(t, rngs, act, 0.25).backward(dy)
    wide, h = [v.detach().double() for v in t], 2.0**-20
    f = lambda at: float((plain(at, rngs, act, 0.25) * dy.double()).sum())
    first = lambda at: ref_drop(at[0], rngs[0]) @ at[1].t() + at[2]  # the activation's inputs
    back = ref_drop(ref_drop(dy.double(), rngs[2]) @ wide[3], rngs[1]).abs()  # its outputs' gradients
    terms = float((plain(wide, rngs, act, 0.25) * dy.double()).abs().sum())
    for k, v in enumerate(t):
        direction = torch.randn(v.shape, device="cuda", generator=gen).double()
        ends = [[(u + s * h * direction) if j == k else u for j, u in enumerate(wide)] for s in (1, -1)]
        slope = (f(ends[0]) - f(ends[1])) / (2 * h)
        along = float((v.grad.double() * direction).sum())
        off = 512 * ref.ULP * float(((v.grad.abs() + v.grad.abs().max()).double() * direction.abs()).sum())
        off += 2.0**-28 * terms
        if act == "relu":
            a, b = first(ends[0]), first(ends[1])
            off += float(((a - b).abs() / (2 * h) * back)[(a > 0) != (b > 0)].sum()) / 2
        assert abs(slope - along) <= off, (act, k)


def ref_drop(v, rng):
    mask, scale = ref.kept(rng.tolist(), 0.25, *v.shape)
    return v * mask.to(v.device) * scale


def step_of(m, n, k, dtype):
    gen = torch.Generator(device="cuda").manual_seed(m + n + k)
    x = torch.randn(m, k, device="cuda", generator=gen).to(dtype)
    w = (torch.randn(n, k, device="cuda", generator=gen) * k**-0.5).to(dtype)
    b, h = torch.randn(n, device="cuda", generator=gen).to(dtype), torch.randn(m, n, device="cuda", generator=gen).to(dtype)
    rng = torch.tensor([5, 6], device="cuda")

    def step(stream=None, rng=rng):
        x1 = cp.dropout(x, 0.1, rng, stream=stream)
        r = cp.linear(x1, w, b, h, "gelu", 0.2, rng, z=True, stream=stream)
        dz, db = cp.linear_act_grad(r.y, r.z, "gelu", 0.2, rng, stream=stream)
        dx = cp.linear_dx(dz, w, dres=x, stream=stream)
        dw = cp.linear_dw(dz, x1, stream=stream)
        more = cp.linear_dw(dz, x, into=dw.clone() if stream is None else cp.linear_dw(dz, x1, stream=stream), stream=stream)
        return [x1, r.y, r.z, dz, db, dx, dw, more]

    return step


# few rows with K over several workgroups, small and large tiles, K in parts, odd rows
SHAPES = [(1, 512, 20000), (9, 300, 500), (200, 136, 3001), (1030, 520, 264), (2048, 8192, 192)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_replayed_from_a_graph(m, n, k, dtype):
    print(f"graph m={m} n={n} k={k} {dtype}", flush=True)
    step = step_of(m, n, k, dtype)
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
            t.fill_(3.0)
        step()  # eager work between replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for j, (t, v) in enumerate(zip(out, want)):
            assert torch.equal(t, v), f"replay {r}, output {j}"
    del graph


def test_two_graphs_and_eager_work_share_no_workspace():
    a, b = step_of(1, 512, 20000, torch.bfloat16), step_of(300, 136, 6000, torch.float32)
    want = [[t.clone() for t in f()] for f in (a, b)]
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for g, f in zip(graphs, (a, b)):
        with torch.cuda.graph(g):
            outs.append(f())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for r in range(REPLAYS):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = a()
        torch.cuda.synchronize()
        for got, w in zip([*outs, eager], [*want, want[0]]):
            assert all(torch.equal(t, v) for t, v in zip(got, w)), r
    del graphs


def test_a_graph_that_moves_its_offset_on():
    x = torch.ones(300, 200, device="cuda")
    rng = torch.tensor([11, 0], device="cuda")
    one = torch.tensor([0, 1], device="cuda")
    cp.dropout(x, 0.5, rng)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rng.add_(one)
        y = cp.dropout(x, 0.5, rng)
    for r in range(1, REPLAYS + 1):
        graph.replay()
        torch.cuda.synchronize()
        assert rng.tolist() == [11, r]
        assert torch.equal(y, cp.dropout(x, 0.5, torch.tensor([11, r], device="cuda")))
    del graph


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_on_another_stream(m, n, k):
    step = step_of(m, n, k, torch.float16)
    want = step()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.memory._record_memory_history(context=None)
    try:
        outs = step(side)
        made = [e for e in torch.cuda.memory._snapshot()["device_traces"][torch.cuda.current_device()] if e["action"] == "alloc"]
    finally:
        torch.cuda.memory._record_memory_history(enabled=None)
    assert len(made) >= 8 and {e["stream"] for e in made} == {side.cuda_stream}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    again = step(side.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, want))


def test_tensors_that_are_written_count_as_changed():
    x, dz = torch.randn(5, 32, device="cuda"), torch.randn(5, 7, device="cuda")
    rng = torch.tensor([1, 2], device="cuda")
    for make, write in ((lambda: torch.zeros(7, 32, device="cuda"), lambda out: cp.linear_dw(dz, x, into=out)),
                        (lambda: torch.zeros(5, 32, device="cuda"), lambda out: cp.dropout(x, 0.5, rng, out=out))):
        out = make()
        for version in (1, 2):
            assert write(out) is out and out._version == version
        saved = torch.ones_like(out)
        y = torch.ones_like(out).requires_grad_() * saved
        write(saved)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()


def test_offsets_past_32_bits():
    """Rows whose bytes lie past 2^31 and 2^32 of their matrix's start."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GiB")
    n, d = 5_000_000, 512
    rng = torch.tensor([1, 2], device="cuda")
    x = torch.ones(n, d, dtype=torch.bfloat16, device="cuda")
    y = cp.dropout(x, 0.5, rng)
    for row in (0, 2_097_152, 4_194_304, n - 1):
        mask = torch.tensor([bool(v) for v in _row_mask(row, d, 0.5, (1, 2))])
        assert torch.equal((y[row] != 0).cpu(), mask), row
    dz, db = cp.linear_act_grad(x, x, act="relu", p=0.5, rng=rng)
    assert torch.equal(dz, y)
    share = 2 * (y != 0).sum(0, dtype=torch.float64)
    assert ((db.double() - share).abs() <= 2.0**-20 * share).all()
    del x, y, dz
    m, k = 1_100_000, 2048  # 4.5 GB of bf16
    x = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    at = [0, 524_288, 1_048_576, m - 1]
    for j, row in enumerate(at):
        x[row, j] = 1.0
    w = torch.randn(16, k, device="cuda").bfloat16()
    out = cp.linear(x, w).y
    for j, row in enumerate(at):
        assert torch.equal(out[row], w[:, j]), row
    assert int((out != 0).any(1).sum()) == len(at)
    back = cp.linear_dw(out, x)
    want = torch.zeros(16, k, dtype=torch.float64, device="cuda")
    for j in range(len(at)):
        want[:, j] = w[:, j].double()
    assert torch.equal(back.double(), want)


def _row_mask(row, d, p, rng):
    import numpy as np

    chunks = np.arange(-(-d // 8), dtype=np.uint64)
    full = lambda v: np.full_like(chunks, v)
    words = ref.philox([chunks, full(row), full(rng[1] & 0xFFFFFFFF), full(rng[1] >> 32)], (rng[0] & 0xFFFFFFFF, rng[0] >> 32))
    halves = np.stack([h for v in words for h in (v & np.uint64(0xFFFF), v >> np.uint64(16))], axis=1).reshape(-1)[:d]
    return halves >= round(65536 * p)
