"""Plain 64-bit forms of the readout's product, its gradients and dropout, for their tests, with how far a 32-bit result
that is rounded once may be from them."""
from __future__ import annotations

import math

import numpy as np
import torch

from ops_reference import HALF

ULP = 2.0**-24
ACTS = [None, "relu", "gelu", "gelu_tanh", "silu"]
TINY = {torch.float32: 2.0**-149, torch.bfloat16: 2.0**-133, torch.float16: 2.0**-24}  # the smallest step


def philox(counter, key):
    """Philox4x32-10 of uint64 arrays that hold 32-bit words."""
    c, k = [np.asarray(v, dtype=np.uint64) for v in counter], list(key)
    low, shift = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> shift) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> shift) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def kept(rng, p, n, d):
    """(mask [n, d], scale) of dropout with rng = (seed, offset)."""
    t = round(65536 * p)
    seed, offset = (int(v) % (1 << 64) for v in rng)
    rows, chunks = np.meshgrid(np.arange(n, dtype=np.uint64), np.arange(-(-d // 8), dtype=np.uint64), indexing="ij")
    words = philox([chunks, rows, np.full_like(rows, offset & 0xFFFFFFFF), np.full_like(rows, offset >> 32)],
                   (seed & 0xFFFFFFFF, seed >> 32))
    halves = np.stack([h for w in words for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))], axis=2)
    return torch.from_numpy((halves.reshape(n, -1)[:, :d] >= t).copy()), 65536.0 / (65536 - t)


def act(z, name):
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z**3))
    return z * torch.sigmoid(z) if name == "silu" else z


def slope(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        r = 2 * math.sqrt(2 / math.pi)
        g = torch.sigmoid(r * (z + 0.044715 * z**3))
        return g + z * g * (1 - g) * r * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        g = torch.sigmoid(z)
        return g + z * g * (1 - g)
    return torch.ones_like(z)


def rounding(t, dtype):
    """Half a step of dtype at each value."""
    return t.abs() * HALF[dtype] + TINY[dtype]


def linear(x, w, bias, residual, name, p, rng):
    """(y, z) and how far each may be off: k steps of 2^-24 of the sum of magnitudes in z, 1.13 (the largest slope) times
    that and 16 steps in the activation, the scale's and the residual's roundings, and the output's own."""
    dtype, k = x.dtype, x.shape[1]
    x, w = x.double(), w.double()
    z, s = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        z, s = z + bias.double(), s + bias.double().abs()
    off = (k + 2) * ULP * s
    a = act(z, name)
    off_a = 1.13 * off + 16 * ULP * (1 + z.abs()) if name else off
    if p:
        mask, scale = kept(rng.tolist(), p, *z.shape)
        a, off_a = torch.where(mask.to(a.device), a * scale, torch.zeros_like(a)), off_a * scale
    y, mag = a, a.abs()
    if residual is not None:
        y, mag = a + residual.double(), a.abs() + residual.double().abs()
    off_y = off_a + 4 * ULP * mag
    return y, z, off_y + rounding(y.abs() + off_y, dtype), off + rounding(z.abs() + off, dtype)


def act_grad(dy, z, name, p, rng):
    """(dz, db) and how far each may be off: the slope by 16 steps (1 + z^2, as its argument's error counts z-fold and z is
    exact), the products' roundings, dz's own; db by a step of each of its partial sums."""
    dtype = dy.dtype
    dy = dy.double()
    sl = slope(z.double(), name) if name else torch.ones_like(dy)
    dz = dy * sl
    off = dy.abs() * 16 * ULP * (2 + (sl.abs() if name else 0))
    if p:
        mask, scale = kept(rng.tolist(), p, *dz.shape)
        mask = mask.to(dz.device)
        dz, off = torch.where(mask, dz * scale, torch.zeros_like(dz)), torch.where(mask, off * scale, torch.zeros_like(dz))
    off_db = off.sum(0) + (dz.shape[0] + 2) * ULP * dz.abs().sum(0) + TINY[torch.float32]
    return dz, dz.sum(0), off + rounding(dz.abs() + off, dtype), off_db


def product(a, b, dtype, add=None):
    """a @ b, plus add, and how far a 32-bit sum rounded to dtype may be off."""
    a, b = a.double(), b.double()
    y, s = a @ b, a.abs() @ b.abs()
    if add is not None:
        y, s = y + add.double(), s + add.double().abs()
    off = (a.shape[1] + 2) * ULP * s
    return y, off + rounding(y.abs() + off, dtype)


def assert_near(got, want, off, what=""):
    top = torch.finfo(got.dtype).max * (1 + HALF[got.dtype])  # from here on the nearest value is infinity
    got = got.double()
    assert got.shape == want.shape, what
    bad = ~((got - want).abs() <= off) & ~(torch.isinf(got) & (got.sign() == want.sign()) & (want.abs() + off >= top))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: " \
                          f"{float(got[bad][0])} for {float(want[bad][0])} within {float(off[bad][0])}"
