"""Plans and gradients about the sizes at which a plan changes from one
workgroup to several, and about the length at which a row's run is split."""
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


def batches(kind, n, rows, gen):
    if kind == "same":
        return torch.full((n,), rows - 1, dtype=torch.int64)
    if kind == "none":
        return torch.randint(rows, 2**62, (n,), generator=gen)
    if kind == "padded":
        ids = torch.randint(0, rows, (n,), generator=gen)
        ids[torch.rand(n, generator=gen) < 0.4] = -1
        return ids
    return torch.arange(n).remainder(rows).flip(0)


@pytest.mark.parametrize("n", [1, 63, 65, 1023, 1025, 4095, 4096, 4097, 32_768, 32_769])
@pytest.mark.parametrize("rows", [1, 511, 512, 100_000, 2**33])
@pytest.mark.parametrize("kind", ["same", "none", "padded", "descending"])
def test_plan(n, rows, kind):
    print(f"plan n={n} rows={rows} {kind}", flush=True)
    ids = batches(kind, n, rows, torch.Generator().manual_seed(n))
    plan = cp.embed_plan(ids.cuda(), rows)
    order = torch.sort(ids, stable=True).indices
    order = order[(ids[order] >= 0) & (ids[order] < rows)]
    unique, slot, counts = torch.unique_consecutive(ids[order], return_inverse=True, return_counts=True)
    u, v = unique.numel(), order.numel()
    assert int(plan.count) == u
    assert torch.equal(plan.order[:v].cpu().long(), order) and torch.equal(plan.slot[:v].cpu().long(), slot)
    assert (plan.slot[v:] == -1).all()
    assert torch.equal(plan.unique[:u].cpu(), unique)
    assert plan.starts[:u + 1].tolist() == [0] + torch.cumsum(counts, 0).tolist()


@pytest.mark.parametrize("length", [1, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 400])
@pytest.mark.parametrize("n", [3000, 200_000])
def test_gradient_of_runs_of_one_length(length, n):
    print(f"runs of {length}, n={n}", flush=True)
    rows, d = n // length + 1, 24
    ids = torch.arange(n, device="cuda") // length
    dout = torch.randint(-4, 5, (n, d), device="cuda", generator=torch.Generator(device="cuda").manual_seed(n)).float()
    want = torch.zeros(rows + 1, d, dtype=torch.float64, device="cuda").index_add_(0, ids, dout.double())[:rows]
    shuffled = torch.randperm(n, generator=torch.Generator().manual_seed(length)).cuda()
    plan = cp.embed_plan(ids[shuffled], rows)
    whole = cp.embed_grad(plan, dout[shuffled])
    assert torch.equal(whole.double(), want)  # whole numbers: exact in any order
    some = cp.embed_grad_rows(plan, dout[shuffled])
    assert torch.equal(some[:int(plan.count)], whole[plan.unique[:int(plan.count)]])
