"""The 8-bit quantiser at rows and columns of more values than one launch has
threads for: every scale and value against the definition, on the GPU."""
from __future__ import annotations

import pytest
import torch

import trellis_coded_row_amd as cp

pytestmark = pytest.mark.gpu
PART = 2**27  # values checked at a time


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    torch.cuda.init()
    yield
    torch.cuda.empty_cache()


def scaled(x, e):
    """x / 2^e, the power of two from its bits."""
    return x * ((127 - e) << 23).to(torch.int32).view(torch.float32)


def definition(x):
    """(values, scales) of a vector, both as bytes: groups of 128, the least power of two with |x| / scale <= 448."""
    g = torch.nn.functional.pad(x.float(), (0, -x.numel() % 128)).view(-1, 128)
    fraction, exponent = torch.frexp(g.abs().amax(1))
    e = exponent - 9 + (fraction > 0.875)
    q = scaled(g, e[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(-1)[:x.numel()]
    return q, (e + 127).to(torch.uint8)


def filled(*shape):
    return torch.full(shape, 0x5A, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("d", [2**30, 2**30 + 130, 2**31 - 1])
@pytest.mark.parametrize("blocks", [0, 1])
def test_one_long_row(d, blocks):
    print(f"row of {d}, blocks {blocks}", flush=True)
    x = torch.empty(d, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    groups = -(-d // 128)
    q, s = filled(d + -d % 16), filled(groups + 3)
    r = cp.cp_quantize_fp8(x.data_ptr(), cp.CP_DTYPE_BF16, 1, d, d, blocks, q.data_ptr(), q.numel(), s.data_ptr(),
                           s.numel(), None, 16, None, 1, torch.cuda.current_stream().cuda_stream)
    assert r == cp.CP_OK
    for lo in range(0, d, PART):
        want, scale = definition(x[lo:lo + PART])
        assert torch.equal(q[lo:lo + want.numel()], want) and torch.equal(s[lo // 128:lo // 128 + scale.numel()], scale), lo
    assert (q[d:] == 0x5A).all() and (s[groups:] == 0x5A).all()


def test_one_long_row_transposed():
    # the transposed form's rows are 16 bytes apart, one value in each
    d = 2**29 + 2**20 + 77  # more than one launch's columns
    x = torch.empty(d, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(2))
    groups = -(-d // 128)
    q, s, qt, st = filled(d + -d % 16), filled(groups), filled(d, 16), filled(d)
    r = cp.cp_quantize_fp8(x.data_ptr(), cp.CP_DTYPE_BF16, 1, d, d, 0, q.data_ptr(), q.numel(), s.data_ptr(), groups,
                           qt.data_ptr(), 16, st.data_ptr(), 1, torch.cuda.current_stream().cuda_stream)
    assert r == cp.CP_OK
    for lo in range(0, d, PART):
        part = x[lo:lo + PART]
        want, scale = definition(part)
        assert torch.equal(q[lo:lo + want.numel()], want) and torch.equal(s[lo // 128:lo // 128 + scale.numel()], scale), lo
        fraction, exponent = torch.frexp(part.float().abs())  # each value is a group of its own
        e = torch.where(part != 0, exponent - 9 + (fraction > 0.875), torch.zeros_like(exponent))
        assert torch.equal(st[lo:lo + part.numel()], (e + 127).to(torch.uint8)), lo
        alone = scaled(part.float(), e).to(torch.float8_e4m3fn).view(torch.uint8)
        assert torch.equal(qt[lo:lo + part.numel(), 0], alone), lo
    assert all((qt[lo:lo + PART, 1:] == 0x5A).all() for lo in range(0, d, PART))


def test_one_long_column():
    n = 2**29 + 2**20 + 77
    x = torch.empty(n, 1, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(3))
    q, s, qt, st = filled(n, 16), filled(n), filled(n + -n % 16), filled(-(-n // 128))
    r = cp.cp_quantize_fp8(x.data_ptr(), cp.CP_DTYPE_BF16, n, 1, 1, 0, q.data_ptr(), 16, s.data_ptr(), 1, qt.data_ptr(),
                           qt.numel(), st.data_ptr(), st.numel(), torch.cuda.current_stream().cuda_stream)
    assert r == cp.CP_OK
    for lo in range(0, n, PART):
        want, scale = definition(x[lo:lo + PART, 0])
        assert torch.equal(qt[lo:lo + want.numel()], want), lo
        assert torch.equal(st[lo // 128:lo // 128 + scale.numel()], scale), lo
