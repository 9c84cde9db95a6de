"""The readout's product with its epilogue, and the two products of its backward pass, against plain 64-bit forms."""
from __future__ import annotations

import math

import pytest
import torch

import linear_reference as ref
import trellis_coded_row_amd as cp

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]
# one value, one row, ends inside a chunk of 16 bytes, a step of k, a tile; rows of whole chunks; one step, odd numbers of
# steps, k in parts; tiles of each size
SIZES = [(1, 1, 1), (1, 7, 13), (2, 64, 8), (1, 200, 4096), (5, 33, 700), (8, 128, 24576), (16, 70, 1032), (17, 65, 130),
         (40, 100, 72), (64, 64, 64), (65, 129, 200), (100, 1000, 40), (130, 72, 1000), (257, 300, 96), (300, 520, 4100),
         (1000, 258, 1030)]
LARGE = [(4, 1000, 6000), (3, 70, 20001), (4, 5000, 300), (2048, 8192, 192), (4000, 4104, 328), (1030, 1000, 5000)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    torch.cuda.init()


def normal(gen, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, device="cuda", generator=gen) * scale).to(dtype)


def layer(m, n, k, dtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(m * 7 + n * 3 + k + seed)
    return (normal(gen, m, k, dtype=dtype), normal(gen, n, k, dtype=dtype, scale=k**-0.5), normal(gen, n, dtype=dtype),
            normal(gen, m, n, dtype=dtype), torch.randint(-(1 << 62), 1 << 62, (2,), device="cuda", generator=gen))


@pytest.mark.parametrize("m,n,k", SIZES + LARGE)
@pytest.mark.parametrize("dtype", TYPES)
def test_linear(m, n, k, dtype):
    print(f"linear m={m} n={n} k={k} {dtype}", flush=True)
    x, w, bias, residual, rng = layer(m, n, k, dtype)
    name = ref.ACTS[(m + n + k) % 5]
    for b, r, a, p, z in ((None, None, None, 0.0, False), (bias, residual, name, 0.1, True)):
        got = cp.linear(x, w, bias=b, residual=r, act=a, p=p, rng=rng, z=z)
        y, wide, off_y, off_z = ref.linear(x, w, b, r, a, p, rng)
        ref.assert_near(got.y, y, off_y, "y")
        assert (got.z is not None) == z
        if z:
            ref.assert_near(got.z, wide, off_z, "z")


@pytest.mark.parametrize("m,n,k", SIZES + LARGE)
@pytest.mark.parametrize("dtype", TYPES)
def test_dx(m, n, k, dtype):
    print(f"dx m={m} n={n} k={k} {dtype}", flush=True)
    x, w, _, dz, _ = layer(m, n, k, dtype)
    for dres in (None, x):
        dx = cp.linear_dx(dz, w, dres=dres)
        assert dx.dtype == dtype
        ref.assert_near(dx, *ref.product(dz, w, dtype, dres), "dx")


@pytest.mark.parametrize("m,n,k", SIZES + LARGE)
@pytest.mark.parametrize("dtype", TYPES)
def test_dw(m, n, k, dtype):
    print(f"dw m={m} n={n} k={k} {dtype}", flush=True)
    x, _, _, dz, _ = layer(m, n, k, dtype)
    dw = cp.linear_dw(dz, x)
    assert dw.dtype == torch.float32
    want, off = ref.product(dz.t(), x, torch.float32)
    ref.assert_near(dw, want, off, "dw")
    before = dw.clone()
    assert cp.linear_dw(dz, x, into=dw) is dw
    ref.assert_near(dw, want + before.double(), off + want.abs() * 2 * ref.ULP, "dw added")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name", ref.ACTS)
def test_every_activation(name, dtype):
    """Pre-activations from far below to far above 0, and their gradient."""
    m, n = 37, 200
    z = torch.linspace(-30, 30, m * n, device="cuda").view(m, n).to(dtype)
    one = torch.eye(m, device="cuda").to(dtype)
    y, wide, off_y, _ = ref.linear(one, z.t().contiguous(), None, None, name, 0.0, None)
    ref.assert_near(cp.linear(one, z.t().contiguous(), act=name).y, y, off_y, name)
    dy = torch.ones_like(z)
    dz, db = cp.linear_act_grad(dy, z, act=name)
    want, sums, off, off_db = ref.act_grad(dy, z, name, 0.0, None)
    ref.assert_near(dz, want, off, "dz")
    ref.assert_near(db, sums, off_db, "db")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name", ["relu", "gelu", "gelu_tanh", "silu"])
def test_infinities_and_nan(name, dtype):
    z = torch.tensor([[float("inf"), -float("inf"), float("nan"), 0.0, -0.0, 60000.0, -60000.0, 1.0]], device="cuda").to(dtype)
    y = cp.linear(torch.ones(1, 0, device="cuda", dtype=dtype), torch.ones(8, 0, device="cuda", dtype=dtype), bias=z[0],
                  act=name).y[0].tolist()
    assert y[0] == math.inf and y[1] == 0 and math.isnan(y[2]) and y[3] == y[4] == 0 and y[6] == 0
    assert y[5] == float(z[0, 5])
    dz, db = cp.linear_act_grad(torch.ones_like(z), z, act=name)
    dz = dz[0].tolist()
    assert dz[0] == 1 and dz[1] == 0 and dz[5] == 1 and dz[6] == 0
    assert dz[2] == 0 if name == "relu" else math.isnan(dz[2])
    assert dz[3] == dz[4] == (0 if name == "relu" else 0.5)
    assert db[:2].tolist() == [1, 0]


def test_a_value_that_is_not_finite_stays_in_its_row():
    """Nothing past an end of a row, or in a row beside it, enters a sum."""
    for dtype in TYPES:
        for m, n, k in ((70, 70, 70), (300, 200, 1031), (9, 100, 520), (130, 136, 264)):
            x, w, _, dz, _ = layer(m, n, k, dtype)
            big = torch.full((m + 2, k + 8), float("nan"), device="cuda", dtype=dtype)
            big[1:m + 1, :k] = x
            wide = torch.full((n + 2, k + 16), float("inf"), device="cuda", dtype=dtype)
            wide[1:n + 1, :k] = w
            back = torch.full((m + 2, n + 8), float("nan"), device="cuda", dtype=dtype)
            back[1:m + 1, :n] = dz
            x2, w2, dz2 = big[1:m + 1, :k], wide[1:n + 1, :k], back[1:m + 1, :n]
            assert torch.equal(cp.linear(x2, w2).y, cp.linear(x2.clone(), w2.clone()).y)
            ref.assert_near(cp.linear(x2, w2).y, *ref.linear(x, w, None, None, None, 0.0, None)[::2], "y")
            ref.assert_near(cp.linear_dx(dz2, w2), *ref.product(dz, w, dtype), "dx")
            ref.assert_near(cp.linear_dw(dz2, x2), *ref.product(dz.t(), x, torch.float32), "dw")
            x2[3, 2] = float("nan")
            got = cp.linear(x2, w2).y
            assert torch.isnan(got[3]).all() and torch.isfinite(got[:3]).all() and torch.isfinite(got[4:]).all()


@pytest.mark.parametrize("over", [1, 2, 5, 7])
@pytest.mark.parametrize("dtype", TYPES)
def test_a_tile_of_less_than_a_chunk(over, dtype):
    """Rows at odd places whose last tile has fewer columns than 16 bytes hold: of 64, 128 and 256 columns."""
    for m, n, k in ((70, 64 + over, 128 + over), (1000, 2048 + over, 1024 + over), (2048 + over, 8192 + over, 200),
                    (3000, 256 + over, 4096 + over)):
        print(f"chunk m={m} n={n} k={k} {dtype}", flush=True)
        x, w, _, dz, _ = layer(m, n, k, dtype)
        ref.assert_near(cp.linear(x, w).y, *ref.linear(x, w, None, None, None, 0.0, None)[::2], "y")
        ref.assert_near(cp.linear_dx(dz, w), *ref.product(dz, w, dtype), "dx")
        ref.assert_near(cp.linear_dw(dz, x), *ref.product(dz.t(), x, torch.float32), "dw")


def test_rows_that_overlap_and_odd_strides():
    for dtype in TYPES:
        x, w, bias, residual, _ = layer(90, 110, 300, dtype)
        row = x[:1].expand(90, 300)
        ref.assert_near(cp.linear(row, w, residual=residual[:1].expand(90, 110)).y,
                        *ref.linear(row, w, None, residual[:1].expand(90, 110), None, 0.0, None)[::2], "one row")
        ref.assert_near(cp.linear_dw(residual[:1].expand(90, 110), row),
                        *ref.product(residual[:1].expand(90, 110).t(), row, torch.float32), "dw of one row")
        ref.assert_near(cp.linear_dx(residual, w[:1].expand(110, 300)),
                        *ref.product(residual, w[:1].expand(110, 300), dtype), "dx of one row")
        flat = torch.randn(90 * 307 + 300, device="cuda").to(dtype)
        for start in (0, 1, 3, 8):
            odd = flat[start:start + 90 * 306].as_strided((90, 300), (305, 1), start)
            ref.assert_near(cp.linear(odd, w).y, *ref.linear(odd, w, None, None, None, 0.0, None)[::2], "odd stride")


def test_no_columns_no_rows():
    for dtype in TYPES:
        x, w, bias, residual, rng = layer(6, 10, 16, dtype)
        for act in ref.ACTS:
            got = cp.linear(x[:, :0], w[:, :0], bias=bias, residual=residual, act=act, p=0.5, rng=rng, z=True)
            y, z, off_y, off_z = ref.linear(x[:, :0], w[:, :0], bias, residual, act, 0.5, rng)
            ref.assert_near(got.y, y, off_y, "y")
            ref.assert_near(got.z, z, off_z, "z")
        assert cp.linear(x[:0], w, bias=bias).y.shape == (0, 10) and cp.linear(x, w[:0]).y.shape == (6, 0)
        assert (cp.linear_dx(residual[:, :0], w[:0], dres=x) == x).all() and cp.linear_dx(residual[:0], w).shape == (0, 16)
        assert (cp.linear_dw(residual[:0], x[:0]) == 0).all() and cp.linear_dw(residual, x[:, :0]).shape == (10, 0)
        into = torch.ones(10, 16, device="cuda")
        assert (cp.linear_dw(residual[:0], x[:0], into=into) == 1).all()
        dz, db = cp.linear_act_grad(residual[:0], residual[:0], act="silu")
        assert dz.shape == (0, 10) and (db == 0).all()


@pytest.mark.parametrize("m,n,k", [(1, 40, 64), (9, 40, 64), (70, 130, 72), (300, 264, 33), (2048, 8192, 64)])
@pytest.mark.parametrize("dtype,tiny,large", [(torch.float32, 2.0**-140, 2.0**100), (torch.bfloat16, 2.0**-130, 2.0**100),
                                              (torch.float16, 2.0**-22, 2.0**9)])
def test_values_below_the_smallest_normal_one(m, n, k, dtype, tiny, large):
    """Their products with large ones are exact, few and small whole multiples of tiny times large."""
    gen = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randint(-3, 4, (m, k), device="cuda", generator=gen).double()
    w = torch.randint(-2, 3, (n, k), device="cuda", generator=gen).double()
    d = torch.randint(-1, 2, (m, n), device="cuda", generator=gen).double()
    want = (x @ w.t() * tiny * large).float()
    assert torch.equal(cp.linear((x * tiny).to(dtype), (w * large).to(dtype)).y, want.to(dtype))
    assert torch.equal(cp.linear_dx((d * large).to(dtype), (w * tiny).to(dtype)), (d @ w * tiny * large).float().to(dtype))
    assert torch.equal(cp.linear_dw((d * large).to(dtype), (x * tiny).to(dtype)), (d.t() @ x * tiny * large).float())


def test_into_rows_of_a_wider_matrix():
    x, _, _, dz, _ = layer(50, 20, 72, torch.bfloat16)
    wide = torch.full((22, 80), 5.0, device="cuda")
    part = wide[1:21, 3:75]
    cp.linear_dw(dz, x, into=part)
    want, off = ref.product(dz.t(), x, torch.float32)
    ref.assert_near(part, want + 5.0, off + 20 * ref.ULP, "part")
    wide[1:21, 3:75] = 5.0
    assert (wide == 5.0).all()


@pytest.mark.parametrize("m,n,k", [(8, 300, 2000), (700, 264, 3000), (2100, 1100, 72)])
@pytest.mark.parametrize("dtype", TYPES)
def test_equal_calls_give_equal_bits(m, n, k, dtype):
    x, w, bias, residual, rng = layer(m, n, k, dtype)
    calls = [lambda: cp.linear(x, w, bias, residual, "gelu", 0.3, rng).y, lambda: cp.linear_dx(residual, w),
             lambda: cp.linear_dw(residual, x), lambda: cp.linear_act_grad(residual, residual, "silu")[1]]
    for call in calls:
        first = call()
        for _ in range(3):
            assert torch.equal(call(), first)
