"""The 8-bit quantiser and product against plain 64-bit forms. The quantiser
is exact: scales and values are compared for equality. The product of k
values a b: k steps of 2^-24 of the sum of magnitudes, and for 16-bit outputs
the rounding and the matrix instruction's cut-off (2^-16 of a group's largest
product, at most, for each of its 8 products: within 2^-13 of the sum)."""
from __future__ import annotations

import math

import pytest
import torch

import trellis_coded_row_amd as cp
from ops_reference import HALF, block_scales, groups, on_grid, row_scales, same, spread, values

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    torch.cuda.init()


def matrix(n, d, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, d, generator=g) * torch.exp(torch.randn(n, 1, generator=g))).to(dtype)


def check_rows(x, q, scale):
    n, d = x.shape
    s = row_scales(x.double())
    assert (scale.cpu().double() == s).all()
    assert same(q.cpu().double(), on_grid(x.double() / spread(s, n, d)))


@pytest.mark.parametrize("n,d", [(1, 1), (3, 127), (128, 128), (129, 257), (1, 1000), (300, 17), (127, 640), (1000, 130)])
@pytest.mark.parametrize("dtype", TYPES)
def test_quantize(n, d, dtype):
    print(f"quantize n={n} d={d} {dtype}", flush=True)
    x = matrix(n, d, n + d, dtype)
    q, scale, qt, st = cp.quantize_fp8(x.cuda(), transposed=True)
    check_rows(x, q, scale)
    check_rows(x.t().contiguous(), qt, st)
    q2, scale2, none, none_t = cp.quantize_fp8(x.cuda())
    assert none is None and none_t is None
    assert same(q2.float(), q.float()) and (scale2.float() == scale.float()).all()
    b, bs, bt, bst = cp.quantize_fp8(x.cuda(), blocks=True, transposed=True)
    s = block_scales(x.double())
    assert (bs.cpu().double() == s).all() and (bst.cpu().double() == s.t()).all()
    assert same(b.cpu().double(), on_grid(x.double() / spread(s, n, d, 128)))
    assert same(bt.cpu().double(), b.cpu().double().t())
    b2, bs2, _, _ = cp.quantize_fp8(x.cuda(), blocks=True)
    assert same(b2.float(), b.float()) and (bs2.float() == bs.float()).all()


def test_quantize_special_values():
    x = torch.zeros(6, 300)
    x[0, 0], x[0, 1], x[0, 2] = math.inf, -math.nan, -3.0      # take no part in the scale
    x[1, 5] = 448.0                                            # exactly the largest value
    x[2, 5] = math.nextafter(448.0, 500.0) + 2.0**-15          # just past it: the next scale
    x[3, 5] = 2.0**-149                                        # the least subnormal: the least scale
    x[4, 130] = 3.0e38
    x[4, 131] = -1.0e-30
    x[5, :] = torch.linspace(-1, 1, 300)                       # ties and every sign
    x[5, 7] = -0.0
    q, scale, qt, st = cp.quantize_fp8(x.cuda(), transposed=True)
    check_rows(x, q, scale)
    check_rows(x.t().contiguous(), qt, st)
    assert float(scale[1, 0]) == 1.0 and float(scale[2, 0]) == 2.0 and float(scale[3, 0]) == 2.0**-127
    assert torch.isnan(q[0, :2].float()).all() and float(scale[0, 1]) == 1.0
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    x = torch.where(torch.isnan(every), torch.zeros(256), every)[None, :].repeat(2, 1)
    q, scale, _, _ = cp.quantize_fp8(x.cuda())                 # every e4m3 value stays itself
    assert (q.float().cpu() * spread(scale.cpu().float(), 2, 256) == x).all()


def test_quantize_views_and_bytes_past_the_rows():
    big = matrix(200, 700, 5).cuda()
    x = big[3:190, 11:450]
    q, scale, qt, st = cp.quantize_fp8(x, transposed=True)
    check_rows(x.cpu(), q, scale)
    check_rows(x.cpu().t().contiguous(), qt, st)
    n, d = 5, 133
    x = matrix(n, d, 6).cuda()
    q = torch.full((n, 160), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.full((n, 7), 0x33, dtype=torch.uint8, device="cuda")
    qt = torch.full((d, 16), 0x5A, dtype=torch.uint8, device="cuda")
    st = torch.full((d, 3), 0x33, dtype=torch.uint8, device="cuda")
    r = cp.cp_quantize_fp8(x.data_ptr(), cp.CP_DTYPE_F32, n, d, d, 0, q.data_ptr(), 160, s.data_ptr(), 7, qt.data_ptr(),
                           16, st.data_ptr(), 3, torch.cuda.current_stream().cuda_stream)
    assert r == cp.CP_OK
    assert (q[:, d:] == 0x5A).all() and (s[:, 2:] == 0x33).all() and (qt[:, n:] == 0x5A).all() and (st[:, 1:] == 0x33).all()
    check_rows(x.cpu(), q[:, :d].contiguous().view(torch.float8_e4m3fn), s[:, :2].contiguous().view(torch.float8_e8m0fnu))
    for a, b in ((0, 5), (5, 0)):
        q, s, qt, st = cp.quantize_fp8(torch.empty(a, b, device="cuda"), transposed=True)
        assert q.shape == (a, b) and qt.shape == (b, a)


def operands(m, n, k, blocks, seed, poison=True):
    """8-bit operands; the bytes past each row's end are NaN."""
    a, sa, _, _ = cp.quantize_fp8(matrix(m, k, seed).cuda())
    b, sb, _, _ = cp.quantize_fp8(matrix(n, k, seed + 1).cuda(), blocks=blocks)
    if poison:
        for t in (a, b):
            if t.shape[1] % 16 and t.shape[0]:
                whole = t.as_strided((t.shape[0], -(-t.shape[1] // 16) * 16), (t.stride(0), 1)).view(torch.uint8)
                whole[:, t.shape[1]:] = 0x7F
        for t in (sa, sb):
            if t.shape[1] % 4 and t.shape[0]:
                whole = t.as_strided((t.shape[0], -(-t.shape[1] // 4) * 4), (t.stride(0), 1)).view(torch.uint8)
                whole[:, t.shape[1]:] = 0xFF
    return a, sa, b, sb


def within(out, want, tol):
    """|out - want| <= tol, or the type's infinity where want may round past its largest value."""
    over = torch.isinf(out) & (torch.sign(out.double()) == torch.sign(want)) & (
        want.abs() + tol > torch.finfo(out.dtype).max)
    return ((out.double() - want).abs() <= tol) | over


def check_product(a, sa, b, sb, out, blocks):
    k = a.shape[1]
    x, y = values(a, sa), values(b, sb, 128 if blocks else 1)
    want, mags = x @ y.t(), x.abs() @ y.abs().t()
    tol = mags * (k + 2) * 2.0**-24
    if out.dtype != torch.float32:
        tol = tol + mags * 2.0**-13 + want.abs() * HALF[out.dtype] + 2.0**-25
    bad = ~within(out.cpu(), want, tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, first at {torch.nonzero(bad)[0].tolist()}"


@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 64, 128), (3, 17, 130), (8, 200, 4096), (16, 33, 1000), (17, 300, 520),
                                   (40, 129, 777), (64, 16, 2048), (65, 65, 129), (100, 64, 5000), (128, 128, 128),
                                   (200, 130, 384), (129, 257, 1023), (300, 700, 640), (513, 260, 2049),
                                   (700, 1030, 1152)])
@pytest.mark.parametrize("blocks", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
def test_product(m, n, k, blocks, dtype):
    print(f"product m={m} n={n} k={k} blocks={blocks} {dtype}", flush=True)
    a, sa, b, sb = operands(m, n, k, blocks, m + n + k)
    out = cp.gemm_fp8(a, sa, b, sb, dtype=dtype)
    check_product(a, sa, b, sb, out, blocks)
    assert torch.equal(out, cp.gemm_fp8(a, sa, b, sb, dtype=dtype))


@pytest.mark.parametrize("m,n,k", [(2048, 2048, 512), (1500, 4100, 640), (4096, 2048, 136)])
@pytest.mark.parametrize("dtype", TYPES)
def test_large_products(m, n, k, dtype):
    # against torch's product of the widened operands in 64 bits, on the GPU
    print(f"product m={m} n={n} k={k} {dtype}", flush=True)
    a, sa, b, sb = operands(m, n, k, False, m + n + k)
    out = cp.gemm_fp8(a, sa, b, sb, dtype=dtype)
    x = a.double() * sa.double().repeat_interleave(128, 1)[:, :k]
    y = b.double() * sb.double().repeat_interleave(128, 1)[:, :k]
    want, mags = x @ y.t(), x.abs() @ y.abs().t()
    tol = mags * (k + 2) * 2.0**-24
    if dtype != torch.float32:
        tol = tol + mags * 2.0**-13 + want.abs() * HALF[dtype] + 2.0**-25
    assert within(out, want, tol).all()


def test_every_place_of_the_operands_is_multiplied_once():
    # one-hot rows: out[i][j] = a[i][p_i] b[j][p_i], so a value in the wrong place shows
    for m, n, k in ((48, 80, 300), (200, 96, 300), (300, 300, 512)):
        g = torch.Generator().manual_seed(m)
        p = torch.randint(0, k, (m,), generator=g)
        x = torch.zeros(m, k)
        x[torch.arange(m), p] = torch.randint(1, 8, (m,), generator=g).float()
        y = torch.randint(-8, 9, (n, k), generator=g).float()
        one = lambda t: torch.full((t.shape[0], groups(k)), 127, dtype=torch.uint8)
        pad = lambda t, u: torch.nn.functional.pad(t, (0, -t.shape[1] % u))
        qa = pad(x, 16).to(torch.float8_e4m3fn).cuda()[:, :k]
        qb = pad(y, 16).to(torch.float8_e4m3fn).cuda()[:, :k]
        sa = pad(one(x), 4).cuda().view(torch.float8_e8m0fnu)[:, :groups(k)]
        sb = pad(one(y), 4).cuda().view(torch.float8_e8m0fnu)[:, :groups(k)]
        for dtype in TYPES:
            print(f"one-hot m={m} n={n} k={k} {dtype}", flush=True)
            assert (cp.gemm_fp8(qa, sa, qb, sb, dtype=dtype).float().cpu() == x @ y.t()).all()


def test_scales_reach_over_their_whole_range():
    m, n, k = 80, 96, 256
    for ea, eb in ((-60, 60), (-110, 100), (110, -115), (-127, 100), (3, 5)):
        a, sa, b, sb = operands(m, n, k, False, 7)
        sa.view(torch.uint8).fill_(127 + ea)
        sb.view(torch.uint8).fill_(127 + eb)
        print(f"scales 2^{ea} and 2^{eb}", flush=True)
        out = cp.gemm_fp8(a, sa, b, sb, dtype=torch.bfloat16)
        check_product(a, sa, b, sb, out, False)
        if ea > -124:
            check_product(a, sa, b, sb, cp.gemm_fp8(a, sa, b, sb, dtype=torch.float32), False)
    a, sa, b, sb = operands(m, n, k, False, 8)
    sa.view(torch.uint8)[5, 1] = 255  # NaN: that row alone
    for dtype in TYPES:
        out = cp.gemm_fp8(a, sa, b, sb, dtype=dtype)
        assert torch.isnan(out[5]).all() and torch.isfinite(out[torch.arange(m) != 5]).all()
    a, sa, b, sb = operands(m, n, k, False, 9)
    b.view(torch.uint8)[7, 200] = 0x7F  # a NaN value: that column alone
    for dtype in TYPES:
        out = cp.gemm_fp8(a, sa, b, sb, dtype=dtype)
        assert torch.isnan(out[:, 7]).all() and torch.isfinite(out[:, torch.arange(n) != 7]).all()


def test_product_views_outputs_and_refusals():
    m, n, k = 70, 90, 200
    a, sa, b, sb = operands(m, n, k, False, 3)
    want = cp.gemm_fp8(a, sa, b, sb)
    big = torch.full((m, 200), 7.0, dtype=torch.bfloat16, device="cuda")
    cp.gemm_fp8(a, sa, b, sb, out=big[:, 50:50 + n])  # a view: its neighbours stay
    assert torch.equal(big[:, 50:50 + n], want) and (big[:, :50] == 7).all() and (big[:, 50 + n:] == 7).all()
    wide = torch.zeros(m, 512, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    wide[:, 32:32 + k] = a
    assert torch.equal(cp.gemm_fp8(wide[:, 32:32 + k], sa, b, sb), want)
    nothing = cp.gemm_fp8(a[:, :0], sa[:, :0], b[:, :0], sb[:, :0], dtype=torch.float32)
    assert nothing.shape == (m, n) and (nothing == 0).all()
    assert cp.gemm_fp8(a[:0], sa[:0], b, sb).shape == (0, n)
    odd = torch.zeros(m, 201, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    for call in (lambda: cp.gemm_fp8(odd[:, :k], sa, b, sb), lambda: cp.gemm_fp8(wide[:, 33:33 + k], sa, b, sb),
                 lambda: cp.gemm_fp8(a[:, :150], sa, b, sb), lambda: cp.gemm_fp8(a, sa[:, :1], b, sb),
                 lambda: cp.gemm_fp8(a, sa, b, sb[:50]), lambda: cp.gemm_fp8(a, sa, b, sb, dtype=torch.int32),
                 lambda: cp.gemm_fp8(a, sa, b, sb, out=big), lambda: cp.gemm_fp8(a.float(), sa, b, sb),
                 lambda: cp.gemm_fp8(a, sa, b, sb, out=big[:, :n].t())):
        with pytest.raises(ValueError):
            call()


def test_norm_output_feeds_the_product():
    x, w = matrix(130, 1000, 1, torch.bfloat16).cuda(), torch.ones(1000, dtype=torch.bfloat16, device="cuda")
    r = cp.rms_norm(x, w, y=False, fp8=True)
    b, sb, _, _ = cp.quantize_fp8(matrix(300, 1000, 2, torch.bfloat16).cuda(), blocks=True)
    check_product(r.q, r.scale, b, sb, cp.gemm_fp8(r.q, r.scale, b, sb), True)
