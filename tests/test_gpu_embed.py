"""The uncompressed row table's lookup and gradient against plain 64-bit
forms. Tolerances: a 32-bit product and a rounding for the lookup; for a sum
of c terms (c + 2) steps of 2^-24 of the sum of magnitudes."""
from __future__ import annotations

import pytest
import torch

import trellis_coded_row_amd as cp
from ops_reference import HALF

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    torch.cuda.init()


def make_ids(n, rows, seed, bad=True):
    g = torch.Generator().manual_seed(seed)
    u = torch.rand(n, generator=g)
    ids = ((u**4) * rows).long().clamp(max=max(rows - 1, 0))  # low rows often, as in a vocabulary
    if bad and n > 3:
        ids[torch.randperm(n, generator=g)[: max(1, n // 9)]] = -1
        ids[n // 2] = rows
        ids[n // 3] = -(2**40)
    return ids


@pytest.mark.parametrize("d", [1, 7, 8, 64, 100, 511, 512, 1024, 2050])
@pytest.mark.parametrize("n", [1, 5, 777])
def test_lookup_sizes(n, d):
    print(f"lookup n={n} d={d}", flush=True)
    rows = 301
    table = torch.randn(rows, d, generator=torch.Generator().manual_seed(d)).bfloat16()
    ids = make_ids(n, rows, n + d)
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = cp.embed_lookup(table.cuda(), ids.cuda(), scale=1.7, bad_id=bad)
    ok = (ids >= 0) & (ids < rows)
    want = torch.where(ok[:, None], table[ids.clamp(0, rows - 1)].double() * 1.7, torch.zeros(n, d, dtype=torch.float64))
    tol = want.abs() * (HALF[torch.bfloat16] + 3 * 2.0**-24)
    assert ((out.cpu().double() - want).abs() <= tol).all()
    assert int(bad) == int((ids >= rows).any())


@pytest.mark.parametrize("ti", TYPES)
@pytest.mark.parametrize("to", TYPES)
def test_lookup_types_strides_and_large_batches(ti, to):
    n, rows, d = 40_001, 513, 65
    big = torch.randn(rows, 2 * d + 3, generator=torch.Generator().manual_seed(4)).to(ti).cuda()
    table = big[:, 3:3 + d]  # rows neither contiguous nor aligned
    ids = make_ids(n, rows, 9).cuda()
    print(f"lookup {ti} -> {to}", flush=True)
    out = cp.embed_lookup(table, ids, scale=0.3, dtype=to)
    ok = (ids >= 0) & (ids < rows)
    scale = float(torch.tensor(0.3))
    want = torch.where(ok[:, None], table[ids.clamp(0, rows - 1)].double() * scale, 0.0)
    assert ((out.double() - want).abs() <= want.abs() * (HALF[to] + 2.0**-24) + 2.0**-25).all()  # fp16 subnormals


def test_lookup_of_an_empty_batch_table_and_row():
    t = torch.randn(4, 8, device="cuda")
    assert cp.embed_lookup(t, torch.empty(0, dtype=torch.int64, device="cuda")).shape == (0, 8)
    none = torch.empty(0, 8, device="cuda")
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = cp.embed_lookup(none, torch.tensor([0, -1], device="cuda"), bad_id=bad)
    assert (out == 0).all() and int(bad) == 1
    assert cp.embed_lookup(torch.empty(3, 0, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")).shape == (2, 0)
    # infinities and NaN are values like others; rows of zeros for padding all the same
    t[1, 0], t[1, 1] = float("inf"), float("nan")
    out = cp.embed_lookup(t, torch.tensor([1, -1], device="cuda"), scale=2.0)
    assert torch.isinf(out[0, 0]) and torch.isnan(out[0, 1]) and (out[1] == 0).all()


def test_lookup_past_32_bit_offsets():
    rows, d = 5_000_011, 512  # 5.1 GB, 2.56e9 elements
    table = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 4_194_303, 4_194_304, 8_388_607 // 2, rows - 1, 4_500_001])
    table[at.cuda()] = torch.arange(1, 7, dtype=torch.bfloat16, device="cuda")[:, None]
    out = cp.embed_lookup(table, at.cuda())
    assert (out == table[at.cuda()]).all()


def check_plan(plan, ids, rows):
    ids = ids.cpu()
    ok = (ids >= 0) & (ids < rows)
    keep = torch.nonzero(ok)[:, 0]
    order = keep[torch.sort(ids[keep], stable=True).indices]
    unique, inverse, counts = torch.unique(ids[order], return_inverse=True, return_counts=True)
    u = int(plan.count)
    assert u == unique.numel()
    assert (plan.unique[:u].cpu() == unique).all()
    assert (plan.order[: order.numel()].cpu().long() == order).all()
    assert (plan.slot[: order.numel()].cpu().long() == inverse).all()
    starts = torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(counts, 0)])
    assert (plan.starts[: u + 1].cpu().long() == starts).all()


@pytest.mark.parametrize("n", [0, 1, 2, 63, 64, 1000, 1024, 1025, 4096, 5000, 16384, 16385, 60_001])
@pytest.mark.parametrize("rows", [0, 1, 500, 131072, 97_690_000, 2**32, 2**32 + 5, 2**61])
def test_plan(n, rows):
    print(f"plan n={n} rows={rows}", flush=True)
    g = torch.Generator().manual_seed(n + rows % 97)
    if rows == 0:
        ids = torch.randint(-3, 3, (n,), generator=g)
    elif rows > 2**31:
        ids = torch.randint(0, rows, (n,), generator=g)
        if n > 2:
            ids[: n // 2] = ids[n // 2: 2 * (n // 2)]  # each twice
            ids[n // 2] = rows
            ids[-1] = rows - 1
    else:
        ids = make_ids(n, rows, n)
    ids = ids.cuda()
    check_plan(cp.embed_plan(ids, rows), ids, rows)


@pytest.mark.parametrize("kind", ["same", "descending", "all_bad", "two"])
@pytest.mark.parametrize("n", [3000, 40_000, 300_000])
def test_plan_of_unusual_batches(kind, n):
    rows = 1_000_000
    print(f"plan {kind} n={n}", flush=True)
    ids = {"same": torch.full((n,), 77), "descending": torch.arange(n, 0, -1), "all_bad": torch.full((n,), -1),
           "two": torch.arange(n) % 2 * (rows - 1)}[kind].cuda()
    check_plan(cp.embed_plan(ids, rows), ids, rows)


def grad_reference(ids, dout, scale, rows):
    """(rows' ids, 64-bit gradient, its tolerance) of the lookups in [0, rows)."""
    ids, dout = ids.cpu(), dout.cpu().double()
    keep = torch.nonzero((ids >= 0) & (ids < rows))[:, 0]
    unique, inverse, counts = torch.unique(ids[keep], return_inverse=True, return_counts=True)
    g = torch.zeros(unique.numel(), dout.shape[1], dtype=torch.float64).index_add_(0, inverse, dout[keep])
    m = torch.zeros_like(g).index_add_(0, inverse, dout[keep].abs())
    s = float(torch.tensor(scale))
    return unique, g * s, m * s * (counts[:, None] + 2) * 2.0**-24


@pytest.mark.parametrize("n,rows,d", [(1, 5, 8), (48, 1000, 512), (777, 40, 33), (5000, 300, 64), (5000, 3, 130),
                                      (20_000, 9000, 1024), (70_000, 700, 65), (40_000, 1, 96), (3000, 2000, 1)])
@pytest.mark.parametrize("dtype", TYPES)
def test_gradient(n, rows, d, dtype):
    print(f"gradient n={n} rows={rows} d={d} {dtype}", flush=True)
    ids = make_ids(n, rows, n + d).cuda()
    dout = torch.randn(n, d, generator=torch.Generator().manual_seed(n)).to(dtype).cuda()
    plan = cp.embed_plan(ids, rows)
    unique, want, tol = grad_reference(ids, dout, 1.3, rows)
    u = unique.numel()
    got = cp.embed_grad_rows(plan, dout, scale=1.3)
    assert int(plan.count) == u and ((got[:u].cpu().double() - want).abs() <= tol).all()
    whole = cp.embed_grad(plan, dout, scale=1.3)
    assert whole.shape == (rows, d)
    full = torch.zeros(rows, d, dtype=torch.float64)
    full[unique] = got[:u].cpu().double()
    assert (whole.cpu().double() == full).all()  # the same sums, zeros elsewhere
    again = cp.embed_grad(plan, dout, scale=1.3)
    assert torch.equal(whole, again)


def test_gradient_of_runs_that_meet_chunk_ends():
    # run lengths around the chunk sizes and the length from which a run is summed in parts
    lengths = [1, 7, 8, 9, 31, 32, 33, 63, 64, 65, 127, 255, 256, 257, 300, 1000, 4097, 2, 64, 64, 64, 256, 256, 1]
    ids = torch.repeat_interleave(torch.arange(len(lengths)) * 3, torch.tensor(lengths))
    for extra in (0, 5, 300_000):  # a larger batch has larger chunks
        tail = torch.randint(100, 300_000, (extra,), generator=torch.Generator().manual_seed(1))
        allids = torch.cat([ids, tail])
        allids = allids[torch.randperm(allids.numel(), generator=torch.Generator().manual_seed(2))].cuda()
        dout = torch.randn(allids.numel(), 40, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
        plan = cp.embed_plan(allids, 300_000)
        unique, want, tol = grad_reference(allids, dout, 1.0, 300_000)
        got = cp.embed_grad_rows(plan, dout)[: unique.numel()]
        print(f"runs, extra={extra}", flush=True)
        assert ((got.cpu().double() - want).abs() <= tol).all()


def test_gradient_strides_broadcast_and_nothing():
    ids = make_ids(500, 50, 3).cuda()
    plan = cp.embed_plan(ids, 50)
    big = torch.randn(500, 77, device="cuda")
    for dout in (big[:, 5:70], big[:1, :65].expand(500, 65)):  # a view, and one row for all
        unique, want, tol = grad_reference(ids, dout, 1.0, 50)
        got = cp.embed_grad_rows(plan, dout)[: unique.numel()]
        assert ((got.cpu().double() - want).abs() <= tol).all()
    with pytest.raises(ValueError):
        cp.embed_grad(plan, big[:400])
    none = cp.embed_plan(torch.full((5,), -1, dtype=torch.int64, device="cuda"), 50)
    assert int(none.count) == 0 and (cp.embed_grad(none, torch.ones(5, 12, device="cuda")) == 0).all()
    empty = cp.embed_plan(torch.empty(0, dtype=torch.int64, device="cuda"), 50)
    assert int(empty.count) == 0 and (cp.embed_grad(empty, torch.ones(0, 12, device="cuda")) == 0).all()


def test_gradient_keeps_infinities_to_their_rows():
    ids = torch.tensor([3, 1, 3, -1, 2], device="cuda")
    dout = torch.ones(5, 16, device="cuda")
    dout[1, 4], dout[3, :] = float("inf"), float("nan")  # row 1; padding takes no part
    whole = cp.embed_grad(cp.embed_plan(ids, 5), dout)
    assert torch.isinf(whole[1, 4]) and torch.isfinite(whole[[0, 2, 3, 4]]).all()
    assert (whole[3] == 2).all() and (whole[0] == 0).all()


def test_gradient_against_differences():
    # f = sum(c * lookup(T)) is linear in T: a difference quotient is exact up to rounding
    g = torch.Generator().manual_seed(5)
    table, c = torch.randn(20, 9, generator=g), torch.randn(60, 9, generator=g)
    ids = torch.randint(0, 20, (60,), generator=g)
    grad = cp.embed_grad(cp.embed_plan(ids.cuda(), 20), c.cuda(), scale=3.0).cpu()

    def f(t):
        return float((c.double() * cp.embed_lookup(t.cuda(), ids.cuda(), scale=3.0).cpu().double()).sum())

    for r, k in ((0, 0), (7, 3), (19, 8)):
        up, down = table.clone(), table.clone()
        up[r, k] += 0.5
        down[r, k] -= 0.5
        # 60 x 9 products, each rounded once at values up to about 12
        assert abs((f(up) - f(down)) / float(up[r, k].double() - down[r, k].double()) - float(grad[r, k])) < 540 * 12 * 2.0**-23
