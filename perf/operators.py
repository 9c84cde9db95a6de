"""The dense operators on either side of the compressed table, as cases to measure.

A row table is trained uncompressed before its rows are coded: `embed` is the lookup into it, `embed_grad` the gradient
that comes back (whole, for a vocabulary; distinct rows only, for a hashed table). Decoded rows go to the readout:
`norm` is the root-mean-square norm with the residual's addition and an 8-bit output, `norm_grad` its gradient,
`quant` the 8-bit form of weights and gradients, `gemm` the product of two 8-bit operands.

8-bit values are e4m3 with one power-of-two scale (e8m0) for 128 values: for a group with largest finite magnitude A the
scale is the least 2^e with A / 2^e <= 448 (1 where A is 0). Values that are not finite become e4m3's NaN.

Sizes: 48 rows of 512 values per token, 393,216 lookups and 97,690,000 rows are those of this repository's replay;
hidden sizes and vocabularies are round numbers. Where `own` is false everything runs in elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
GROUP = 128
EPS = 1e-6
ZIPF = 1.1
READOUT = 48 * 512  # one token's rows of one memory layer, side by side


# --------------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one decoding step's rows from a table in training: 48 ids, where the call's latency is what counts
        {"name": "embed_step", "op": "embed", "n": 48, "rows": 1 << 20, "d": 512, "type": "bf16", "out": "bf16", "pad": 0.0},
        # the replay's lookups (4,096 tokens, 48 rows, 2 layers) into an uncompressed table
        {"name": "embed_replay", "op": "embed", "n": 393216, "rows": 1 << 22, "d": 512, "type": "bf16", "out": "bf16", "pad": 0.0},
        # a vocabulary's gradient of one batch, padding among its tokens, in the 32 bits that the optimiser reads
        {"name": "embed_grad_vocab", "op": "embed_grad", "n": 16384, "rows": 1 << 17, "d": 1024, "type": "bf16", "whole": True, "pad": 0.1},
        # the replay's gradient for a table of 97,690,000 rows: the distinct rows alone
        {"name": "embed_grad_replay", "op": "embed_grad", "n": 393216, "rows": 97_690_000, "d": 512, "type": "bf16", "whole": False, "pad": 0.0},
        # eight sequences' next tokens between two layers: residual, norm, 8 bits
        {"name": "norm_step", "op": "norm", "n": 8, "d": 4096, "type": "bf16", "residual": True, "eight": True, "sixteen": False},
        # a prompt's looked-up rows before the readout's product
        {"name": "norm_readout", "op": "norm", "n": 4096, "d": READOUT, "type": "bf16", "residual": False, "eight": True, "sixteen": False},
        # training: the gradient of a residual norm, the stream's own gradient added
        {"name": "norm_grad", "op": "norm_grad", "n": 8192, "d": 4096, "type": "bf16", "residual": True},
        # the readout's weight after an update: 128 x 128 blocks, for the product and, transposed, for its gradient
        {"name": "quant_weight", "op": "quant", "n": 4096, "d": READOUT, "type": "bf16", "form": "blocks"},
        # a ragged batch's output gradient: groups along the row, and along the tokens for the weight's gradient
        {"name": "quant_grad_ragged", "op": "quant", "n": 1000, "d": 2050, "type": "bf16", "form": "rows"},
        # the readout for eight sequences' next tokens: the weight is read once
        {"name": "gemm_step", "op": "gemm", "m": 8, "n": 4096, "k": READOUT, "wide": True, "out": "bf16"},
        # the readout for a prompt of 4,096 tokens
        {"name": "gemm_prompt", "op": "gemm", "m": 4096, "n": 4096, "k": READOUT, "wide": True, "out": "bf16"},
        # the readout weight's gradient over those tokens: both operands have a scale for each row's 128 values
        {"name": "gemm_weight_grad", "op": "gemm", "m": 4096, "n": READOUT, "k": 4096, "wide": False, "out": "f32"},
    ]


def _log(rng, lo, hi):
    """A size between lo and hi, spread over the logarithm; none is a multiple of 1,024, which the listed cases are."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return v - (v % 1024 == 0)


def _even(v):
    """A multiple of 128 near v."""
    return v // 256 * 256 + 128


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "quant", "gemm", "gemm"])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("embed", "embed_grad"):
        d = rng.choice([64, 128, 256, 512, _log(rng, 32, 1024)])
        n = _log(rng, 1, 393216 * 512 // max(d, 512))
        pad = rng.choice([0.0, 0.05, 0.3])
        if op == "embed":
            return {"op": op, "n": n, "rows": _log(rng, 1000, 1 << 21), "d": d, "type": kind,
                    "out": rng.choice(["bf16", kind]), "pad": pad}
        whole = rng.random() < 0.5
        return {"op": op, "n": n, "rows": _log(rng, 500, (1 << 27) // d) if whole else _log(rng, 1000, 97_690_000), "d": d,
                "type": kind, "whole": whole, "pad": pad}
    if op in ("norm", "norm_grad", "quant"):
        d = _log(rng, 64, READOUT)
        d = rng.choice([d, min(_even(d), READOUT)])
        n = _log(rng, 1, min(16384, 4096 * 4096 // d if op == "norm_grad" else 4096 * READOUT // 2 // d))
        if op == "quant":
            return {"op": op, "n": n, "d": d, "type": kind, "form": rng.choice(["rows", "blocks"])}
        c = {"op": op, "n": n, "d": d, "type": kind, "residual": rng.random() < 0.6}
        if op == "norm":
            eight, sixteen = rng.choice([(True, False), (True, True), (False, True)])
            c.update(eight=eight, sixteen=sixteen)
        return c
    k, n = _log(rng, 128, READOUT), _log(rng, 64, 8192)
    m = _log(rng, 1, max(1, min(8192, 4096 * 4096 * READOUT // 4 // (n * k))))
    if rng.random() < 0.6:
        k, n = _even(k), _even(n)
    return {"op": op, "m": m, "n": n, "k": k, "wide": rng.random() < 0.6, "out": rng.choice(["bf16", "f16", "f32"])}


# -------------------------------------------------------------------------------------------------------- the inputs

def _ids(n, rows, pad, gen):
    """n row ids, Zipf-distributed over scattered rows; a share `pad` of them is padding (-1). How often the most
    frequent row comes, the next one and so on is the same for each seed, so that the number of distinct rows is too;
    which rows those are, and where in the batch they stand, goes by the seed."""
    valid = n - int(n * pad)
    u = torch.rand(valid, dtype=torch.float64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(n))
    top = 1.0 - (rows + 1.0) ** (1.0 - ZIPF)
    rank = ((1.0 - u * top) ** (1.0 / (1.0 - ZIPF))).long().clamp(1, rows) - 1
    first = torch.randint(rows, (1,), device="cuda", generator=gen)
    ids = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    ids[:valid] = (rank * 2654435761 + first) % rows  # a prime above every table's size: each rank has a row of its own
    return ids[torch.randperm(n, device="cuda", generator=gen)]


def _distinct(n, rows):
    """The expected number of distinct rows among n of _ids' lookups."""
    top = 1.0 - (rows + 1.0) ** (1.0 - ZIPF)
    edge = np.unique(np.floor(np.exp(np.linspace(0.0, math.log(rows + 1.0), 4000))))
    wide = np.diff(edge)
    share = -np.diff(edge ** (1.0 - ZIPF)) / top
    return max(1.0, float(np.sum(wide * -np.expm1(-n * share / wide))))


def _normal(gen, *shape):
    return torch.randn(*shape, device="cuda", generator=gen)


def _activations(gen, n, d):
    """Activations: a few columns far above the others, as hidden states have them."""
    return _normal(gen, n, d).mul_(torch.exp(_normal(gen, d) * 0.7))


def _padded(rows, cols, dtype):
    """An empty rows x cols matrix of 8-bit values whose rows start on 16 bytes."""
    return torch.empty(rows, (cols + 15) // 16 * 16, dtype=dtype, device="cuda")[:, :cols]


def _eight_bits(gen, n, k, wide):
    """e4m3 values [n, k] and e8m0 scales of a normal matrix: a scale for 128 values of a row, or for 128 x 128."""
    x = _normal(gen, n, k).mul_(torch.exp(_normal(gen, n, 1)))
    q, s = _blocks(x) if wide else _rows(x)
    out, groups = _padded(n, k, torch.float8_e4m3fn), s.shape[1]
    out.copy_(q)
    scale = torch.zeros(s.shape[0], (groups + 3) // 4 * 4, dtype=torch.uint8, device="cuda")
    scale[:, :groups] = s.view(torch.uint8)
    return out, scale.view(torch.float8_e8m0fnu)[:, :groups]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 11)
    op, c = case["op"], case
    if op in ("embed", "embed_grad"):
        s = {"ids": _ids(c["n"], c["rows"], c["pad"], gen)}
        kind = TYPES[c["type"]]
        if op == "embed":
            s["table"] = torch.empty(c["rows"], c["d"], dtype=kind, device="cuda").normal_(generator=gen).mul_(0.02)
        else:
            s["dout"] = _normal(gen, c["n"], c["d"]).mul_(0.01).to(kind)
    elif op in ("norm", "norm_grad"):
        kind = TYPES[c["type"]]
        s = {"x": _activations(gen, c["n"], c["d"]).to(kind), "weight": (1 + 0.2 * _normal(gen, c["d"])).to(kind)}
        if op == "norm_grad":
            x = s["x"].float()
            s["rstd"] = torch.rsqrt((x * x).mean(1) + EPS)
            s["dy"] = _normal(gen, c["n"], c["d"]).mul_(0.01).to(kind)
            s["dres"] = _normal(gen, c["n"], c["d"]).mul_(0.01).to(kind) if c["residual"] else None
        else:
            s["residual"] = _activations(gen, c["n"], c["d"]).to(kind) if c["residual"] else None
    elif op == "quant":
        s = {"x": _activations(gen, c["n"], c["d"]).mul_(0.02).to(TYPES[c["type"]])}
    else:
        s = {}
        s["a"], s["a_scale"] = _eight_bits(gen, c["m"], c["k"], False)
        s["b"], s["b_scale"] = _eight_bits(gen, c["n"], c["k"], c["wide"])
    s["case"] = dict(case)
    return s


# ---------------------------------------------------------------------------------------------------- the plain forms

def _scale_of(amax):
    """The least power of two 2^e with amax / 2^e <= 448 = 0.875 * 2^9, within e8m0's range; 1 for amax = 0."""
    fraction, exponent = torch.frexp(amax)  # amax = fraction * 2^exponent, fraction in [0.5, 1)
    e = (exponent - 9 + (fraction > 0.875)).clamp(-127, 127)
    return torch.where(amax > 0, e, torch.zeros_like(e))


def _to_e4m3(x, e):
    """x / 2^e in e4m3; what is not finite becomes NaN. (No 32-bit value needs an e above 120: 2^-e is a normal number.)"""
    q = x * ((127 - e) << 23).to(torch.int32).view(torch.float32)
    return torch.where(torch.isfinite(x), q, torch.full_like(q, math.nan)).to(torch.float8_e4m3fn)


def _finite(x):
    return torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))


def _e8m0(e):
    return (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _fill(x, rows, cols):
    """x with zeros below and to the right, up to whole groups."""
    return torch.nn.functional.pad(x, (0, -x.shape[1] % cols, 0, -x.shape[0] % rows))


def _rows(x):
    n, d = x.shape
    g = _fill(x, 1, GROUP).view(n, -1, GROUP)
    e = _scale_of(_finite(g).amax(2))
    return _to_e4m3(g, e[:, :, None]).view(n, -1)[:, :d], _e8m0(e)


def _blocks(x):
    n, d = x.shape
    g = _fill(x, GROUP, GROUP)
    g = g.view(g.shape[0] // GROUP, GROUP, -1, GROUP)
    e = _scale_of(_finite(g).amax((1, 3)))
    return _to_e4m3(g, e[:, None, :, None]).view(g.shape[0] * GROUP, -1)[:n, :d], _e8m0(e)


def _widen(q, scale, tall):
    """The 32-bit values of e4m3 q with scales for 128 values of a row (tall 1) or for 128 x 128 (tall 128)."""
    s = scale.to(torch.float32).repeat_interleave(GROUP, 1)[:, : q.shape[1]]
    return q.to(torch.float32) * (s.repeat_interleave(tall, 0)[: q.shape[0]] if tall > 1 else s)


def _plain(s, c):
    op = c["op"]
    if op == "embed":
        ids = s["ids"]
        x = s["table"][ids.clamp(min=0)].float() * math.sqrt(c["d"])
        return torch.where((ids >= 0)[:, None], x, torch.zeros_like(x)).to(TYPES[c["out"]])
    if op == "embed_grad":
        ids, dout = s["ids"], s["dout"].float() * math.sqrt(c["d"])
        if c["whole"]:
            g = torch.zeros(c["rows"] + 1, c["d"], device=ids.device)
            return g.index_add_(0, torch.where(ids >= 0, ids, torch.full_like(ids, c["rows"])), dout)[: c["rows"]]
        rows, place = torch.unique(ids, return_inverse=True)
        g = torch.zeros(rows.shape[0], c["d"], device=ids.device).index_add_(0, place, dout)
        first = int(rows[0] < 0) if c["pad"] else 0
        return {"rows": rows[first:], "grad": g[first:]}
    if op == "norm":
        kind, w = TYPES[c["type"]], s["weight"].float()
        h = s["x"].float()
        out = {}
        if c["residual"]:
            h = h + s["residual"].float()
            out["h"] = h.to(kind)
        rstd = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
        y = h * rstd * w
        out["rstd"] = rstd[:, 0]
        if c["sixteen"]:
            out["y"] = y.to(kind)
        if c["eight"]:
            out["q"], out["scale"] = _rows(y)
        return out
    if op == "norm_grad":
        kind, x, w, dy, rstd = TYPES[c["type"]], s["x"].float(), s["weight"].float(), s["dy"].float(), s["rstd"][:, None]
        hat = x * rstd
        g = dy * w
        dx = rstd * (g - hat * (g * hat).mean(1, keepdim=True))
        if c["residual"]:
            dx = dx + s["dres"].float()
        return {"dx": dx.to(kind), "dw": (dy * hat).sum(0)}
    if op == "quant":
        x = s["x"].float()
        if c["form"] == "blocks":
            q, scale = _blocks(x)
            return {"q": q, "scale": scale, "qt": q.t().contiguous()}
        q, scale = _rows(x)
        qt, scale_t = _rows(x.t().contiguous())
        return {"q": q, "scale": scale, "qt": qt, "scale_t": scale_t}
    a, b = _widen(s["a"], s["a_scale"], 1), _widen(s["b"], s["b_scale"], GROUP if c["wide"] else 1)
    return (a @ b.t()).to(TYPES[c["out"]])


# ------------------------------------------------------------------------------------------------ the framework's calls

def _ours(s, c):
    import trellis_coded_row_amd as cp

    op = c["op"]
    if op == "embed":
        return cp.embed_lookup(s["table"], s["ids"], scale=math.sqrt(c["d"]), dtype=TYPES[c["out"]])
    if op == "embed_grad":
        plan = cp.embed_plan(s["ids"], c["rows"])
        if c["whole"]:
            return cp.embed_grad(plan, s["dout"], scale=math.sqrt(c["d"]))
        grad = cp.embed_grad_rows(plan, s["dout"], scale=math.sqrt(c["d"]))
        u = int(plan.count)  # the number of distinct rows, which sizes what the optimiser does next
        return {"rows": plan.unique[:u], "grad": grad[:u]}
    if op == "norm":
        r = cp.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, y=c["sixteen"], fp8=c["eight"], rstd=True)
        out = {"rstd": r.rstd}
        if c["residual"]:
            out["h"] = r.h
        if c["sixteen"]:
            out["y"] = r.y
        if c["eight"]:
            out["q"], out["scale"] = r.q, r.scale
        return out
    if op == "norm_grad":
        dx, dw = cp.rms_norm_grad(s["dy"], s["x"], s["rstd"], s["weight"], dres=s["dres"])
        return {"dx": dx, "dw": dw}
    if op == "quant":
        if c["form"] == "blocks":
            q, scale, qt, _ = cp.quantize_fp8(s["x"], blocks=True, transposed=True)
            return {"q": q, "scale": scale, "qt": qt}
        q, scale, qt, scale_t = cp.quantize_fp8(s["x"], transposed=True)
        return {"q": q, "scale": scale, "qt": qt, "scale_t": scale_t}
    return cp.gemm_fp8(s["a"], s["a_scale"], s["b"], s["b_scale"], dtype=TYPES[c["out"]])


def run(state):
    return _ours(state, state["case"]) if own else _plain(state, state["case"])


# ------------------------------------------------------------------------------------------------------ what it takes

def work(case):
    c, op = case, case["op"]
    if op in ("embed", "embed_grad"):
        valid = c["n"] * (1 - c["pad"])
        distinct = _distinct(valid, c["rows"])
        es = SIZE[c["type"]]
        if op == "embed":
            return {"bytes": 8 * c["n"] + distinct * c["d"] * es + c["n"] * c["d"] * SIZE[c["out"]], "flops": valid * c["d"]}
        wrote = c["rows"] * c["d"] * 4 if c["whole"] else distinct * (c["d"] * 4 + 8)
        return {"bytes": 8 * c["n"] + valid * c["d"] * es + wrote, "flops": 2 * valid * c["d"]}
    if op in ("norm", "norm_grad", "quant"):
        cells, es = c["n"] * c["d"], SIZE[c["type"]]
        groups = -(-c["d"] // GROUP)
        if op == "norm":
            moved = cells * es * (3 if c["residual"] else 1) + cells * es * c["sixteen"] + (cells + c["n"] * groups) * c["eight"]
            return {"bytes": moved + c["d"] * es + 4 * c["n"], "flops": 5 * cells}
        if op == "norm_grad":
            return {"bytes": cells * es * (4 if c["residual"] else 3) + c["d"] * (es + 4) + 4 * c["n"], "flops": 10 * cells}
        return {"bytes": cells * (es + 2), "flops": 2 * cells}
    cells = c["m"] * c["k"] + c["n"] * c["k"]
    return {"bytes": cells + cells // GROUP + c["m"] * c["n"] * SIZE[c["out"]], "flops": 2 * c["m"] * c["n"] * c["k"]}


# ------------------------------------------------------------------------------------------- the definitions, in 64 bits

def _exact_rows(y):
    """(e4m3 values, scales) of float64 rows, by the definition: the scale by search over whole exponents, the value by
    rounding to e4m3's grid (3 bits below the leading one, steps of 2^-9 under 2^-6), ties to even."""
    n, d = y.shape
    groups = -(-d // GROUP)
    wide = torch.zeros(n, groups * GROUP, dtype=torch.float64, device=y.device)
    wide[:, :d] = torch.where(torch.isfinite(y), y, 0.0)
    top = wide.view(n, groups, GROUP).abs().max(2).values
    guess = torch.floor(torch.log2(torch.clamp(top, min=1e-300) / 448.0)) - 1
    for _ in range(3):  # log2's rounding may leave the guess one off
        guess = torch.where(top > 448.0 * _two_to(guess), guess + 1, guess)
    scale = torch.where(top > 0, _two_to(guess.clamp(-127, 127)), 1.0)
    q = _on_grid(wide.view(n, groups, GROUP) / scale[:, :, None]).view(n, -1)[:, :d]
    return torch.where(torch.isfinite(y), q, torch.nan), scale


def _two_to(e):
    """2^e in 64 bits for whole e, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _on_grid(v):
    """64-bit values within e4m3's range, rounded to its values."""
    exponent = (v.abs().clamp(min=2.0 ** -6).view(torch.int64) >> 52) - 1023
    return torch.round(v / _two_to(exponent - 3)) * _two_to(exponent - 3)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    op = c["op"]
    if op == "embed":
        out = torch.zeros(c["n"], c["d"], dtype=torch.float64, device="cuda")
        at = s["ids"] >= 0
        out[at] = s["table"][s["ids"][at]].double() * c["d"] ** 0.5
        return out
    if op == "embed_grad":
        order = torch.sort(s["ids"], stable=True)
        ids, at = order.values, order.indices
        at, ids = at[ids >= 0], ids[ids >= 0]
        rows, count = torch.unique_consecutive(ids, return_counts=True)
        end = torch.cumsum(count, 0)
        grad = torch.empty(rows.shape[0], c["d"], dtype=torch.float64, device="cuda")
        for lo in range(0, c["d"], 128):  # running sums over the sorted tokens, a slice of the columns at a time
            part = s["dout"][:, lo:lo + 128][at].double() * c["d"] ** 0.5
            run_ = torch.cat([torch.zeros(1, part.shape[1], dtype=torch.float64, device="cuda"), torch.cumsum(part, 0)])
            grad[:, lo:lo + 128] = run_[end] - run_[end - count]
        if not c["whole"]:
            return {"rows": None, "grad": grad}
        out = torch.zeros(c["rows"], c["d"], dtype=torch.float64, device="cuda")
        out[rows] = grad
        return out
    if op == "norm":
        h = s["x"].double() + (s["residual"].double() if c["residual"] else 0.0)
        root = torch.sqrt(torch.sum(h * h, 1) / c["d"] + EPS)
        y = h / root[:, None] * s["weight"].double()
        out = {"rstd": 1.0 / root}
        if c["residual"]:
            out["h"] = h
        if c["sixteen"]:
            out["y"] = y
        if c["eight"]:
            out["q"], out["scale"] = _exact_rows(y)
        return out
    if op == "norm_grad":
        x, w, dy, r = s["x"].double(), s["weight"].double(), s["dy"].double(), s["rstd"].double()
        dot = torch.sum(dy * w * x, 1) / c["d"]
        dx = (dy * w) * r[:, None] - x * (r ** 3 * dot)[:, None]
        if c["residual"]:
            dx += s["dres"].double()
        return {"dx": dx, "dw": torch.sum(dy * x * r[:, None], 0)}
    if op == "quant":
        x = s["x"].double()
        if c["form"] == "rows":
            q, scale = _exact_rows(x)
            qt, scale_t = _exact_rows(x.t().contiguous())
            return {"q": q, "scale": scale, "qt": qt, "scale_t": scale_t}
        n, d = x.shape
        rows, cols = -(-n // GROUP), -(-d // GROUP)
        whole = torch.zeros(rows * GROUP, cols * GROUP, dtype=torch.float64, device="cuda")
        whole[:n, :d] = x
        # a block's magnitudes in one group: the group's scale is the block's
        top = whole.view(rows, GROUP, cols, GROUP).abs().amax((1, 3))
        _, scale = _exact_rows(top.reshape(-1, 1))
        scale = scale.view(rows, cols)
        q = _on_grid(x / scale.repeat_interleave(GROUP, 0)[:n].repeat_interleave(GROUP, 1)[:, :d])
        return {"q": q, "scale": scale, "qt": q.t().contiguous()}
    kb = torch.arange(c["k"], device="cuda") // GROUP
    a = s["a"].double() * s["a_scale"].double()[:, kb]
    tall = torch.arange(c["n"], device="cuda") // (GROUP if c["wide"] else 1)
    b = s["b"].double() * s["b_scale"].double()[tall][:, kb]
    return torch.matmul(a, b.T)
