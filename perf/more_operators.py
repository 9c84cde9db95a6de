"""The readout's product in 16 and 32 bits, its gradients, and dropout, as cases to measure.

Decoded rows of a memory layer go through a product with a bias and an activation and join the residual stream; in
training, dropout is applied to looked-up rows and to the readout. `linear` is the product with all of that in its
epilogue, `act_grad` the gradient back through the epilogue, `dx` and `dw` the two products of the backward pass,
`dropout` the mask on its own. With m tokens, n outputs and k inputs:

    linear    z = x w^T + bias,  y = drop(act(z)) + residual
    act_grad  dz = dy * keep / (1 - p) * act'(z),  db = the sum of dz's rows
    dx        dx = dz w (+ what reaches x past the product)
    dw        dw = dz^T x, in 32 bits
    dropout   y = keep / (1 - p) * x (+ residual)

The mask is never stored: it comes from Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy as
1, 2, 3", 2011) with the key `seed` and the counter (column / 8, row, offset), whose four words are eight halves of 16
bits, low half first, for eight neighbouring columns. A value is kept where its half is at least t = round(65536 p), and
1 / (1 - p) is 65536 / (65536 - t). Seed and offset are an input.

Sizes: 48 rows of 512 values per token and 393,216 lookups are those of this repository's replay; hidden sizes are round
numbers. Where `own` is false everything runs in elementary torch operations.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
READOUT = 48 * 512  # one token's rows of one memory layer, side by side
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


# --------------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one token through a small projection of a memory layer's rows: the call's latency is what counts
        {"name": "linear_token", "op": "linear", "m": 1, "n": 1024, "k": 4096, "type": "bf16", "act": "silu", "bias": True,
         "residual": False, "p": 0.0, "z": False},
        # the readout for eight sequences' next tokens, added to the residual stream: the weight is read once
        {"name": "linear_step", "op": "linear", "m": 8, "n": 4096, "k": READOUT, "type": "bf16", "act": "none", "bias": True,
         "residual": True, "p": 0.0, "z": False},
        # training: the readout of 4,096 tokens, with dropout, the pre-activation kept for the gradient
        {"name": "linear_prompt", "op": "linear", "m": 4096, "n": 4096, "k": READOUT, "type": "bf16", "act": "gelu",
         "bias": True, "residual": True, "p": 0.1, "z": True},
        # a ragged batch through a layer of odd sizes
        {"name": "linear_ragged", "op": "linear", "m": 1000, "n": 2050, "k": 1030, "type": "f16", "act": "gelu_tanh",
         "bias": True, "residual": False, "p": 0.0, "z": False},
        # back through the epilogue of a wide layer over 8,192 tokens
        {"name": "act_grad_wide", "op": "act_grad", "m": 8192, "n": 16384, "type": "bf16", "act": "gelu", "p": 0.1},
        # the same for a ragged batch of a 32-bit layer
        {"name": "act_grad_ragged", "op": "act_grad", "m": 1000, "n": 2050, "type": "f32", "act": "silu", "p": 0.0},
        # the gradient of 4,096 tokens' looked-up rows
        {"name": "dx_prompt", "op": "dx", "m": 4096, "n": 4096, "k": READOUT, "type": "bf16", "residual": False},
        # the same for a ragged batch, with the gradient that came past the layer
        {"name": "dx_ragged", "op": "dx", "m": 1000, "n": 2050, "k": 1030, "type": "f16", "residual": True},
        # the readout weight's gradient over those tokens, in the 32 bits that the optimiser reads
        {"name": "dw_prompt", "op": "dw", "m": 4096, "n": 4096, "k": READOUT, "type": "bf16"},
        # the same for a ragged batch of a 32-bit layer
        {"name": "dw_ragged", "op": "dw", "m": 1000, "n": 2050, "k": 1030, "type": "f32"},
        # dropout of the replay's looked-up rows (4,096 tokens, 48 rows, 2 layers)
        {"name": "dropout_replay", "op": "dropout", "n": 393216, "d": 512, "type": "bf16", "p": 0.1, "residual": False},
        # dropout of a ragged batch on its way into the residual stream
        {"name": "dropout_ragged", "op": "dropout", "n": 1000, "d": 2050, "type": "bf16", "p": 0.3, "residual": True},
    ]


def _log(rng, lo, hi):
    """A size between lo and hi, spread over the logarithm; none is a multiple of 1,024."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return v - (v % 1024 == 0)


def _even(v):
    """A multiple of 64 near v, none of 1,024."""
    return v // 128 * 128 + 64


def draw(rng):
    op = rng.choice(["linear", "linear", "act_grad", "dx", "dw", "dropout"])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    p = rng.choice([0.0, 0.1, 0.2, 0.5])
    if op in ("act_grad", "dropout"):
        d = _log(rng, 64, 16384)
        d = rng.choice([d, _even(d)])
        n = _log(rng, 1, min(65536, (1 << 26) // d))
        if op == "dropout":
            return {"op": op, "n": n, "d": d, "type": kind, "p": p or 0.05, "residual": rng.random() < 0.5}
        return {"op": op, "m": n, "n": d, "type": kind, "act": rng.choice(ACTS[1:]), "p": p}
    k, n = _log(rng, 128, READOUT), _log(rng, 64, 8192)
    m = _log(rng, 1, max(1, min(8192, 4096 * 4096 * READOUT // (16 if kind == "f32" else 4) // (n * k))))
    if rng.random() < 0.6:
        k, n = _even(k), _even(n)
    c = {"op": op, "m": m, "n": n, "k": k, "type": kind}
    if op == "linear":
        c.update(act=rng.choice(ACTS), bias=rng.random() < 0.7, residual=rng.random() < 0.5, p=p, z=rng.random() < 0.4)
    elif op == "dx":
        c["residual"] = rng.random() < 0.4
    return c


# -------------------------------------------------------------------------------------------------------- the inputs

def _normal(gen, *shape):
    return torch.randn(*shape, device="cuda", generator=gen)


def _activations(gen, n, d):
    """Activations: a few columns above the others, as hidden states have them."""
    return _normal(gen, n, d).mul_(torch.exp(_normal(gen, d) * 0.5))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    c, op, kind = case, case["op"], TYPES[case["type"]]
    s = {"case": dict(case)}
    if c.get("p"):
        # (seed, offset) of the generator: any 64 bits
        s["rng"] = torch.randint(-(1 << 62), 1 << 62, (2,), device="cuda", generator=gen)
    if op == "linear":
        s["x"] = _activations(gen, c["m"], c["k"]).to(kind)
        s["w"] = _normal(gen, c["n"], c["k"]).div_(math.sqrt(c["k"])).to(kind)
        s["bias"] = _normal(gen, c["n"]).mul_(0.2).to(kind) if c["bias"] else None
        s["residual"] = _normal(gen, c["m"], c["n"]).to(kind) if c["residual"] else None
    elif op == "act_grad":
        s["dy"] = _normal(gen, c["m"], c["n"]).mul_(0.01).to(kind)
        s["z"] = _normal(gen, c["m"], c["n"]).mul_(1.5).to(kind)
    elif op == "dx":
        s["dz"] = _normal(gen, c["m"], c["n"]).mul_(0.01).to(kind)
        s["w"] = _normal(gen, c["n"], c["k"]).div_(math.sqrt(c["k"])).to(kind)
        s["dres"] = _normal(gen, c["m"], c["k"]).mul_(0.01).to(kind) if c["residual"] else None
    elif op == "dw":
        s["dz"] = _normal(gen, c["m"], c["n"]).mul_(0.01).to(kind)
        s["x"] = _activations(gen, c["m"], c["k"]).to(kind)
    else:
        s["x"] = _activations(gen, c["n"], c["d"]).to(kind)
        s["residual"] = _normal(gen, c["n"], c["d"]).to(kind) if c["residual"] else None
    return s


# ---------------------------------------------------------------------------------------------------- the plain forms

def _philox(c0, c1, offset, seed):
    """Four words of Philox4x32-10 for counters (c0, c1, offset's two halves), as whole numbers in 64 bits."""
    word = 0xFFFFFFFF
    zero = torch.zeros_like(c0 + c1)
    c0, c1, c2, c3 = c0 + zero, c1 + zero, zero + (offset & word), zero + ((offset >> 32) & word)
    k0, k1 = seed & word, (seed >> 32) & word
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # below 2^64: the wrapped product has all its bits
        c0, c1, c2, c3 = (b >> 32) & word ^ c1 ^ k0, b & word, (a >> 32) & word ^ c3 ^ k1, a & word
        k0, k1 = (k0 + 0x9E3779B9) & word, (k1 + 0xBB67AE85) & word
    return c0, c1, c2, c3


def _kept(rng, p, n, d):
    """The mask of an n x d matrix and the scale of what is kept."""
    t = round(65536 * p)
    rows = torch.arange(n, device="cuda")[:, None]
    chunks = torch.arange((d + 7) // 8, device="cuda")[None, :]
    words = torch.stack(_philox(chunks, rows, rng[1], rng[0]), 2)
    halves = torch.stack((words & 0xFFFF, words >> 16), 3).view(n, -1)[:, :d]
    return halves >= t, 65536.0 / (65536 - t)


def _drop(x, s, c):
    if not c["p"]:
        return x
    keep, scale = _kept(s["rng"], c["p"], *x.shape)
    return torch.where(keep, x * scale, torch.zeros_like(x))


def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu":
        return z * 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        r = math.sqrt(2 / math.pi)
        t = torch.tanh(r * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * r * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        g = 1 / (1 + torch.exp(-z))
        return g * (1 + z * (1 - g))
    return torch.ones_like(z)


def _plain(s, c):
    op, kind = c["op"], TYPES[c["type"]]
    if op == "linear":
        z = s["x"].float() @ s["w"].float().t()
        if c["bias"]:
            z = z + s["bias"].float()
        y = _drop(_act(z, c["act"]), s, c)
        if c["residual"]:
            y = y + s["residual"].float()
        return {"y": y.to(kind), "z": z.to(kind)} if c["z"] else {"y": y.to(kind)}
    if op == "act_grad":
        dz = _drop(s["dy"].float() * _slope(s["z"].float(), c["act"]), s, c)
        return {"dz": dz.to(kind), "db": dz.sum(0)}
    if op == "dx":
        dx = s["dz"].float() @ s["w"].float()
        return (dx + s["dres"].float() if c["residual"] else dx).to(kind)
    if op == "dw":
        return s["dz"].float().t() @ s["x"].float()
    y = _drop(s["x"].float(), s, c)
    return (y + s["residual"].float() if c["residual"] else y).to(kind)


# ------------------------------------------------------------------------------------------------ the framework's calls

def _ours(s, c):
    import trellis_coded_row_amd as cp

    op = c["op"]
    act = None if c.get("act") == "none" else c.get("act")
    if op == "linear":
        r = cp.linear(s["x"], s["w"], bias=s["bias"], residual=s["residual"], act=act, p=c["p"], rng=s.get("rng"), z=c["z"])
        return {"y": r.y, "z": r.z} if c["z"] else {"y": r.y}
    if op == "act_grad":
        dz, db = cp.linear_act_grad(s["dy"], s["z"], act=act, p=c["p"], rng=s.get("rng"))
        return {"dz": dz, "db": db}
    if op == "dx":
        return cp.linear_dx(s["dz"], s["w"], dres=s["dres"])
    if op == "dw":
        return cp.linear_dw(s["dz"], s["x"])
    return cp.dropout(s["x"], c["p"], s["rng"], residual=s["residual"])


def run(state):
    return _ours(state, state["case"]) if own else _plain(state, state["case"])


# ------------------------------------------------------------------------------------------------------ what it takes

def work(case):
    c, op, es = case, case["op"], SIZE[case["type"]]
    if op == "dropout":
        return {"bytes": c["n"] * c["d"] * es * (3 if c["residual"] else 2), "flops": c["n"] * c["d"]}
    m, n = c["m"], c["n"]
    if op == "act_grad":
        return {"bytes": 3 * m * n * es + 4 * n, "flops": 10 * m * n}
    k = c["k"]
    flops = 2 * m * n * k
    if op == "linear":
        return {"bytes": es * (m * k + n * k + n * c["bias"] + m * n * (1 + c["residual"] + c["z"])), "flops": flops}
    if op == "dx":
        return {"bytes": es * (m * n + n * k + m * k * (2 if c["residual"] else 1)), "flops": flops}
    return {"bytes": es * (m * n + m * k) + 4 * n * k, "flops": flops}


# ------------------------------------------------------------------------------------------- the definitions, in 64 bits

def _wide_product(x, constant):
    """(high, low) words of a 32-bit x times a 32-bit constant, by 16-bit digits."""
    x0, x1, m0, m1 = x % 65536, x // 65536, constant % 65536, constant // 65536
    mid = x0 * m0 // 65536 + x1 * m0 % 4294967296
    low_mid = mid % 65536 + x0 * m1 % 65536
    high = x1 * m1 + mid // 65536 + x0 * m1 // 65536 + low_mid // 65536
    return high, low_mid % 65536 * 65536 + x0 * m0 % 65536


def _exact_scale(rng, p, n, d):
    """What each value of an n x d matrix is multiplied by: 0, or the scale of what is kept."""
    t = round(p * 65536)
    seed, offset = (int(v) % (1 << 64) for v in rng)
    counter = [torch.arange((d + 7) // 8, device="cuda").repeat(n, 1),
               torch.arange(n, device="cuda").unsqueeze(1).repeat(1, (d + 7) // 8),
               torch.full((n, (d + 7) // 8), offset % (1 << 32), device="cuda"),
               torch.full((n, (d + 7) // 8), offset >> 32, device="cuda")]
    for r in range(10):
        keys = [((seed % (1 << 32)) + r * 0x9E3779B9) % (1 << 32), ((seed >> 32) + r * 0xBB67AE85) % (1 << 32)]
        h0, l0 = _wide_product(counter[0], 0xD2511F53)
        h1, l1 = _wide_product(counter[2], 0xCD9E8D57)
        counter = [torch.bitwise_xor(torch.bitwise_xor(h1, counter[1]), keys[0]), l1,
                   torch.bitwise_xor(torch.bitwise_xor(h0, counter[3]), keys[1]), l0]
    out = torch.empty(n, d, dtype=torch.float64, device="cuda")
    for j in range(min(8, d)):  # the columns whose place among their eight is j
        half = counter[j // 2] // (65536 if j % 2 else 1) % 65536
        out[:, j::8] = (half[:, : (d - j + 7) // 8] >= t).double() * (65536.0 / (65536.0 - t))
    return out


def _exact_act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "gelu":
        return z / 2 * torch.special.erfc(-z / 2 ** 0.5)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * z * (1 + 0.044715 * z ** 2))
    return z * torch.sigmoid(z) if act == "silu" else z


def _exact_slope(z, act):
    """d act / dz by the product and chain rules."""
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return torch.special.erfc(-z / 2 ** 0.5) / 2 + z * torch.exp(-z ** 2 / 2) / (2 * math.pi) ** 0.5
    if act == "gelu_tanh":  # z g(u), u = 2 r (z + 0.044715 z^3), g the logistic function
        r = (2 / math.pi) ** 0.5
        g = torch.sigmoid(2 * r * (z + 0.044715 * z ** 3))
        return g + z * g * (1 - g) * 2 * r * (1 + 0.134145 * z ** 2)
    if act == "silu":
        g = torch.sigmoid(z)
        return g + z * g * (1 - g)
    return torch.ones_like(z)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    op = c["op"]
    if op == "linear":
        z = torch.matmul(s["x"].double(), s["w"].double().T)
        if c["bias"]:
            z += s["bias"].double()
        y = _exact_act(z, c["act"])
        if c["p"]:
            y = y * _exact_scale(s["rng"], c["p"], c["m"], c["n"])
        if c["residual"]:
            y = y + s["residual"].double()
        return {"y": y, "z": z} if c["z"] else {"y": y}
    if op == "act_grad":
        dz = s["dy"].double() * _exact_slope(s["z"].double(), c["act"])
        if c["p"]:
            dz *= _exact_scale(s["rng"], c["p"], c["m"], c["n"])
        return {"dz": dz, "db": torch.sum(dz, 0)}
    if op == "dx":
        dx = torch.matmul(s["dz"].double(), s["w"].double())
        return dx + s["dres"].double() if c["residual"] else dx
    if op == "dw":
        return torch.matmul(s["dz"].double().T, s["x"].double())
    y = s["x"].double() * _exact_scale(s["rng"], c["p"], c["n"], c["d"])
    return y + s["residual"].double() if c["residual"] else y
