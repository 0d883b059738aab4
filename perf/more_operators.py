"""What is measured of the operators around a gated feed-forward block: rows and columns in
microscaled 4-bit floating point (quantised and read back), the linear layer and the gated
block on such codes, the gated block in emulated fp64 with its gradient, and the clipping of
many gradients to a global norm.

``run`` computes each operator in its plain form (elementary torch operations) or, where
``own`` is set, through the library's entry points."""
import math

import torch

own = False

TYPES = {"float64": torch.float64, "float32": torch.float32, "float16": torch.float16,
         "bfloat16": torch.bfloat16}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
# a block of 32 values along K shares the power of two 2^(scale - 127); code c stands for
# GRID[c % 8] with the sign of bit 3
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token's activations before a projection, and the values they stand for
        {"name": "quant_token", "op": "quant", "rows": 1, "cols": 8192, "axis": 0,
         "type": "bfloat16"},
        # a whole prompt's activations before the down-projection
        {"name": "quant_prompt", "op": "quant", "rows": 4096, "cols": 16384, "axis": 0,
         "type": "bfloat16"},
        # a ragged fp32 gradient along the tokens, as a weight gradient's product takes it
        {"name": "quant_columns_ragged", "op": "quant", "rows": 4099, "cols": 5001, "axis": 1,
         "type": "float32"},
        # one token through a square projection: the bytes of the weights
        {"name": "mx_token", "op": "mx", "m": 1, "n": 8192, "k": 8192, "act": "none",
         "residual": True, "type": "bfloat16"},
        # a whole prompt through an up-projection
        {"name": "mx_prompt", "op": "mx", "m": 4096, "n": 16384, "k": 4096, "act": "gelu",
         "residual": True, "type": "bfloat16"},
        # a small batch of requests through a gated block's first half, odd sizes everywhere
        {"name": "mx_gated_batch_odd", "op": "mx_gated", "m": 37, "n": 4100, "k": 1001,
         "act": "silu", "type": "float16"},
        # and a whole prompt
        {"name": "mx_gated_prompt", "op": "mx_gated", "m": 4096, "n": 8192, "k": 4096,
         "act": "silu", "type": "bfloat16"},
        # the gated block of a small network in emulated fp64: a chain of short launches
        {"name": "gated_64", "op": "gated", "m": 64, "n": 64, "k": 64, "r": 14, "act": "gelu"},
        # of a training batch
        {"name": "gated_batch", "op": "gated", "m": 4096, "n": 8192, "k": 4096, "r": 16,
         "act": "silu"},
        # backward through a ragged one: no size a multiple of any tile
        {"name": "gated_grad_ragged", "op": "gated_grad", "m": 1500, "n": 1025, "k": 1001,
         "r": 16, "act": "silu"},
        # the gradients of a small network in fp64
        {"name": "clip_small", "op": "clip", "blocks": 2, "width": 64, "hidden": 170,
         "type": "float64", "clips": True},
        # and of a stack of blocks in bf16
        {"name": "clip_stack", "op": "clip", "blocks": 10, "width": 2048, "hidden": 8191,
         "type": "bfloat16", "clips": True},
    ]


def _spread(rng, low, high):
    """A size spread over the logarithm of [low, high]: odd, even or a multiple of 64."""
    x = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    kind = rng.randrange(3)
    if kind == 0:
        x |= 1
    elif kind == 1 and x >= 64:
        x -= x % 64
    return max(low, min(high, x))


def draw(rng):
    op = rng.choice(("quant", "mx", "mx", "mx_gated", "mx_gated", "gated", "gated_grad", "clip"))
    if op == "quant":
        case = {"op": op, "rows": _spread(rng, 1, 32768), "cols": _spread(rng, 1, 32768),
                "axis": rng.randrange(2),
                "type": rng.choice(("float64", "float32", "float16", "bfloat16"))}
        while case["rows"] * case["cols"] > 1 << 26:
            case["rows"] = case["rows"] // 2 + 1
        return case
    if op in ("mx", "mx_gated"):
        few = rng.random() < 0.5
        case = {"op": op, "m": _spread(rng, 1, 64) if few else _spread(rng, 64, 8192),
                "n": _spread(rng, 128, 16384), "k": _spread(rng, 64, 16384),
                "act": rng.choice(ACTS),
                "type": rng.choice(("float32", "float16", "bfloat16"))}
        if op == "mx":
            case["residual"] = rng.random() < 0.5
        most = 1 << (38 if op == "mx" else 37)
        while case["m"] * case["n"] * case["k"] > most:
            case["m"] = case["m"] // 2 + 1
        return case
    if op in ("gated", "gated_grad"):
        case = {"op": op, "m": _spread(rng, 16, 4096), "n": _spread(rng, 16, 4096),
                "k": _spread(rng, 16, 4096), "r": rng.choice((14, 16)), "act": rng.choice(ACTS)}
        while case["m"] * case["n"] * case["k"] > 1 << 35:
            case["m"] = case["m"] // 2 + 1
        return case
    case = {"op": op, "blocks": rng.randrange(1, 11), "width": _spread(rng, 16, 2048),
            "type": rng.choice(("float64", "float32", "float16", "bfloat16")),
            "clips": rng.random() < 0.7}
    case["hidden"] = _spread(rng, case["width"], 4 * case["width"])
    most = (1 << 30) // TYPES[case["type"]].itemsize
    while case["blocks"] > 1 and 3 * case["blocks"] * case["width"] * case["hidden"] > most:
        case["blocks"] = case["blocks"] // 2
    return case


def _sizes(case):
    """Shapes of the parameters of a stack of pre-norm gated blocks."""
    w, h = case["width"], case["hidden"]
    return [(w,), (w,), (w, 2 * h), (2 * h,), (h, w), (w,)] * case["blocks"]


def _lines(k):
    """Values of a packed line over an inner dimension k: whole steps of 256."""
    return (k + 255) // 256 * 256


def _power(e, dtype):
    """2^e for -127 <= e <= 127, exactly."""
    table = torch.tensor([2.0 ** i for i in range(-127, 128)], dtype=dtype, device=e.device)
    return table[e + 127]


def _quantise(x):
    """(values on GRID's scale, exponents of the blocks) of lines x, zeros past their end:
    2^e the largest power of two whose quadruple does not exceed the block's maximum,
    values past the grid's end at its end."""
    lines, k = x.shape
    kp = _lines(k)
    v = torch.zeros((lines, kp), dtype=x.dtype, device=x.device)
    v[:, :k] = x
    v = v.view(lines, kp // 32, 32)
    amax = v.abs().amax(2)
    e = torch.frexp(amax)[1] - 3
    e = torch.where(amax > 0, e, -127).clamp(-127, 127)
    v = v * _power(-e, x.dtype)[:, :, None]
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(x.dtype)
    q = ((a / step).round() * step).clamp(max=6.0)
    return torch.where(v < 0, -q, q), e


def _pack(x):
    """Codes, two a byte with the even one low, and scales of the lines of x."""
    q, e = _quantise(x)
    a = q.abs().flatten(1)
    c = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    c |= (q.flatten(1) < 0).to(torch.uint8) << 3
    return c[:, 0::2] | c[:, 1::2] << 4, (e + 127).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)

    op = case["op"]
    s = dict(case)
    if op in ("mx", "mx_gated"):
        m, n, k = case["m"], case["n"], case["k"]
        t = TYPES[case["type"]]
        wide = n if op == "mx" else 2 * n
        # tokens of their own scale with a few large channels; rows of weights of their own
        x = normal(m, k) * torch.exp(0.5 * normal(m, 1))
        x *= torch.where(normal(k) > 2.5, 8.0, 1.0)
        w = normal(wide, k) * torch.exp(0.2 * normal(wide, 1)) / math.sqrt(k)
        s["xq"], s["xs"] = _pack(x)
        s["wq"], s["ws"] = _pack(w)
        s["bias"] = normal(wide).to(t)
        if op == "mx":
            s["res"] = normal(m, n).to(t) if case["residual"] else None
    elif op in ("gated", "gated_grad"):
        m, n, k = case["m"], case["n"], case["k"]
        s["a"] = normal(m, k, dtype=torch.float64)
        s["b"] = normal(k, 2 * n, dtype=torch.float64) / math.sqrt(k)
        if op == "gated":
            s["bias"] = normal(2 * n, dtype=torch.float64)
        else:
            s["dc"] = normal(m, n, dtype=torch.float64)
            s["z"] = normal(m, 2 * n, dtype=torch.float64)
    elif op == "quant":
        t = TYPES[case["type"]]
        wide = torch.float64 if t == torch.float64 else torch.float32
        x = normal(case["rows"], case["cols"], dtype=wide)
        x *= torch.exp(0.5 * normal(case["rows"], 1, dtype=wide))
        x *= torch.where(normal(case["cols"], dtype=wide) > 2.5, 8.0, 1.0)
        s["x"] = x.to(t)
    else:
        t = TYPES[case["type"]]
        wide = torch.float64 if t == torch.float64 else torch.float32
        # gradients whose size differs from tensor to tensor
        s["xs"] = [(normal(*shape, dtype=wide) * (0.02 * 2 ** (i % 5))).to(t)
                   for i, shape in enumerate(_sizes(case))]
        s["outs"] = [torch.empty_like(x) for x in s["xs"]]
        s["max_norm"] = 1.0 if case["clips"] else 1e9
    return s


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) * math.sqrt(0.5 / math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        y = 1 / (1 + torch.exp(-z))
        return y + z * y * (1 - y)
    return torch.ones_like(z)


def _run_own(s):
    import fp64_gemm_emulation_ozk_amd as ozk

    op = s["op"]
    if op == "quant":
        k = s["cols"] if s["axis"] == 0 else s["rows"]
        codes, scales = ozk.ozk_mxfp4_quant(s["x"], s["axis"])
        t = TYPES[s["type"]]
        return ozk.ozk_mxfp4_values(codes, scales, k,
                                    dtype=torch.float32 if t == torch.float16 else t)
    if op == "mx":
        return ozk.ozk_mxfp4_linear(s["xq"], s["xs"], s["wq"], s["ws"], bias=s["bias"],
                                    act=s["act"], residual=s["res"], dtype=TYPES[s["type"]])
    if op == "mx_gated":
        return ozk.ozk_mxfp4_gated(s["xq"], s["xs"], s["wq"], s["ws"], bias=s["bias"],
                                   act=s["act"], dtype=TYPES[s["type"]])
    if op == "gated":
        z = torch.empty((s["m"], 2 * s["n"]), dtype=torch.float64, device="cuda")
        c = ozk.ozk_dgemm_gated(s["a"], s["b"], s["r"], bias=s["bias"], act=s["act"],
                                scaling="norm", preact=z)
        return {"c": c, "z": z}
    if op == "gated_grad":
        da, db, dbias = ozk.ozk_dgemm_gated_grad(s["dc"], s["a"], s["b"], s["r"], s["z"],
                                                 act=s["act"], scaling="norm")
        return {"da": da, "db": db, "dbias": dbias}
    norm, outs = ozk.ozk_clip_norm(s["xs"], s["max_norm"], out=s["outs"])
    return [norm, *outs]


def _decode(codes, scales):
    """fp32 values of packed lines."""
    c = torch.stack((codes & 15, codes >> 4), 2).flatten(1)
    grid = torch.tensor(GRID + tuple(-g for g in GRID), device=codes.device)
    power = _power(scales.int() - 127, torch.float32)
    return grid[c.int()] * power.repeat_interleave(32, dim=1)


def run(state):
    s = state
    if own:
        return _run_own(s)
    op = s["op"]
    if op in ("mx", "mx_gated"):
        z = torch.matmul(_decode(s["xq"], s["xs"]), _decode(s["wq"], s["ws"]).t())
        z = z + s["bias"].float()
        if op == "mx_gated":
            c = _act(z[:, :s["n"]], s["act"]) * z[:, s["n"]:]
        else:
            c = _act(z, s["act"])
            c = c if s["res"] is None else c + s["res"].float()
        return c.to(TYPES[s["type"]])
    if op == "gated":
        z = torch.matmul(s["a"], s["b"]) + s["bias"]
        return {"c": _act(z[:, :s["n"]], s["act"]) * z[:, s["n"]:], "z": z}
    if op == "gated_grad":
        zg, zu = s["z"][:, :s["n"]], s["z"][:, s["n"]:]
        g = torch.cat((s["dc"] * zu * _act_slope(zg, s["act"]), s["dc"] * _act(zg, s["act"])), 1)
        return {"da": torch.matmul(g, s["b"].t()), "db": torch.matmul(s["a"].t(), g),
                "dbias": g.sum(0)}
    t = TYPES[s["type"]]
    wide = torch.float64 if t == torch.float64 else torch.float32
    if op == "quant":
        x = s["x"].to(wide)
        x = x if s["axis"] == 0 else x.t()
        q, e = _quantise(x)
        v = (q * _power(e, wide)[:, :, None]).flatten(1)[:, :x.shape[1]]
        return v.to(torch.float32 if t == torch.float16 else t)
    # sums of many squares in 64 bits
    total = torch.stack([x.double().square().sum() for x in s["xs"]]).sum()
    norm = torch.sqrt(total)
    coef = torch.where(norm > s["max_norm"], s["max_norm"] / norm, 1.0).to(wide)
    return [norm] + [(x.to(wide) * coef).to(t) for x in s["xs"]]


def work(case):
    op = case["op"]
    if op in ("gated", "gated_grad"):
        m, n, k = case["m"], case["n"], case["k"]
        if op == "gated":
            return {"bytes": 8 * (m * k + 2 * k * n + 2 * n + 3 * m * n), "flops": 4 * m * n * k}
        return {"bytes": 8 * (3 * m * n + 2 * m * k + 4 * k * n + 2 * n), "flops": 8 * m * n * k}
    e = TYPES[case["type"]].itemsize
    if op in ("mx", "mx_gated"):
        m, n, k = case["m"], case["n"], case["k"]
        wide = n if op == "mx" else 2 * n
        r = 2 if case.get("residual") else 1
        return {"bytes": (m + wide) * (k + 1) // 2 + (m + wide) * ((k + 31) // 32)
                + e * (wide + r * m * n), "flops": 2 * m * wide * k}
    if op == "quant":
        # in, the codes with their scales, and the values they stand for
        x = case["rows"] * case["cols"]
        return {"bytes": e * x + x // 2 + x // 32 + (4 if case["type"] == "float16" else e) * x,
                "flops": 3 * x}
    x = sum(math.prod(shape) for shape in _sizes(case))
    return {"bytes": 2 * e * x + 8, "flops": 3 * x}


def _exact_act(z, act):
    """The activation and its slope at z."""
    if act == "relu":
        return z.clamp(min=0), torch.heaviside(z, torch.zeros_like(z))
    if act == "gelu":
        p = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * p, p + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        # (1 + tanh u) / 2 is the logistic function of 2 u
        u2 = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z.pow(3))
        p = torch.sigmoid(u2)
        return z * p, p + z * p * (1 - p) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z * z)
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p * (1 + z * (1 - p))
    return z, torch.ones_like(z)


def _exact_product(a, b):
    """a b in 64 bits, the inner dimension in two halves."""
    h = a.shape[1] // 2
    return a[:, h:] @ b[h:] + a[:, :h] @ b[:h]


def _exact_power(e):
    """2^e in 64 bits from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_values(codes, scales):
    """Packed lines by the fields of a code: sign, two bits of exponent, one of mantissa."""
    nibbles = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.int32,
                          device=codes.device)
    nibbles[:, 0::2], nibbles[:, 1::2] = codes % 16, codes // 16
    exp, man = nibbles // 2 % 4, nibbles % 2
    mag = torch.where(exp > 0, (2 + man) * 2 ** (exp - 1).clamp(min=0), man).double() / 2
    sign = 1 - 2 * (nibbles // 8)
    power = _exact_power(scales.int() - 127)
    return (mag * sign).view(*scales.shape, 32).mul(power[:, :, None]).flatten(1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("mx", "mx_gated"):
        n = case["n"]
        z = _exact_product(_exact_values(s["xq"], s["xs"]),
                           _exact_values(s["wq"], s["ws"]).t().contiguous())
        z += s["bias"].double()
        if op == "mx_gated":
            return _exact_act(z[:, :n], case["act"])[0] * z[:, n:]
        c = _exact_act(z, case["act"])[0]
        return c + s["res"].double() if case["residual"] else c
    if op == "gated":
        n = case["n"]
        z = _exact_product(s["a"], s["b"]) + s["bias"]
        return {"c": _exact_act(z[:, :n], case["act"])[0] * z[:, n:], "z": z}
    if op == "gated_grad":
        n = case["n"]
        h, slope = _exact_act(s["z"][:, :n], case["act"])
        g = torch.empty_like(s["z"])
        g[:, :n] = s["z"][:, n:] * slope * s["dc"]
        g[:, n:] = h * s["dc"]
        return {"da": _exact_product(g, s["b"].t().contiguous()),
                "db": _exact_product(s["a"].t().contiguous(), g),
                "dbias": torch.ones(1, g.shape[0], dtype=g.dtype, device=g.device).mm(g)[0]}
    if op == "quant":
        # the nearest of the grid's eight values by the seven midpoints between them, a value
        # on a midpoint to the even code
        x = s["x"].double() if case["axis"] == 0 else s["x"].double().t().contiguous()
        out = torch.empty_like(x)
        grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
        mids = (grid[1:] + grid[:-1]) / 2
        for k0 in range(0, x.shape[1], 32):
            v = x[:, k0:k0 + 32]
            amax = torch.linalg.vector_norm(v, ord=math.inf, dim=1)
            power = _exact_power((torch.frexp(amax)[1] - 3).clamp(min=-127, max=127))
            a = v.abs() / power[:, None]
            low, high = torch.searchsorted(mids, a), torch.searchsorted(mids, a, right=True)
            code = torch.where((low < high) & (low % 2 == 0), low, high)
            out[:, k0:k0 + 32] = torch.copysign(grid[code] * power[:, None], v)
        return out
    # squares in order of size would sum no better here: fp64 holds 2^29 of them to 1e-12
    flat = [torch.linalg.vector_norm(x.double()) for x in s["xs"]]
    norm = torch.linalg.vector_norm(torch.stack(flat))
    coef = torch.clamp(s["max_norm"] / norm, max=1.0)
    return [norm] + [x.double() * coef for x in s["xs"]]
