"""Plain 64-bit forms of the dense operators, on the CPU, for their tests."""
from __future__ import annotations

import math

import torch

GROUP = 128
HALF = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}  # half a rounding step, relative


def groups(n: int) -> int:
    return -(-n // GROUP)


def scale_exponent(top: float) -> int:
    """The least e >= -127 with top <= 448 * 2^e; 0 for top = 0."""
    if top == 0:
        return 0
    e = math.floor(math.log2(top / 448.0)) - 1
    while top > math.ldexp(448.0, e):
        e += 1
    return max(e, -127)


def row_scales(x):
    """float64 [n, groups]: the scale of each 128 values of a row."""
    n, d = x.shape
    out = torch.empty(n, groups(d), dtype=torch.float64)
    for g in range(groups(d)):
        part = x[:, g * GROUP:(g + 1) * GROUP]
        top = torch.where(torch.isfinite(part), part.abs(), torch.zeros_like(part)).amax(1)
        out[:, g] = torch.tensor([math.ldexp(1.0, scale_exponent(float(t))) for t in top], dtype=torch.float64)
    return out


def block_scales(x):
    n, d = x.shape
    out = torch.empty(groups(n), groups(d), dtype=torch.float64)
    for i in range(groups(n)):
        for g in range(groups(d)):
            part = x[i * GROUP:(i + 1) * GROUP, g * GROUP:(g + 1) * GROUP]
            top = torch.where(torch.isfinite(part), part.abs(), torch.zeros_like(part)).max()
            out[i, g] = math.ldexp(1.0, scale_exponent(float(top)))
    return out


def spread(scales, n: int, d: int, tall: int = 1):
    """Scales laid out over the n x d values they belong to."""
    return scales.repeat_interleave(tall, 0)[:n].repeat_interleave(GROUP, 1)[:, :d]


def on_grid(v):
    """64-bit values within e4m3's range, rounded to nearest even on its grid; NaN where not finite."""
    ok = torch.isfinite(v)
    a = torch.where(ok, v, torch.zeros_like(v))
    exponent = torch.floor(torch.log2(a.abs().clamp(min=2.0**-6)))
    step = torch.exp2(exponent - 3)
    return torch.where(ok, torch.round(a / step) * step, torch.full_like(v, math.nan))


def same(a, b) -> bool:
    """Equal element by element, NaN equal to NaN."""
    return bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


def values(q, scale, tall: int = 1):
    """float64 values of an 8-bit matrix with its scales."""
    return q.cpu().double() * spread(scale.cpu().double(), *q.shape, tall)
