"""The gated projection, the layer norm and the 8-bit product with scales per block of 128: what they compute in plain
form, and the cases they are measured on.

They stand in a block of a language model next to the operators of `operators.py`: the gated feed-forward projection
(both products, the activation and their product in one) with its backward pass, the layer norm with the residual's
addition and its backward pass, the quantisation of a matrix or of its transpose in E4M3 with one scale per 1 x 128 or
128 x 128 block, and the product of two such matrices.  `run` computes them with elementary torch operations in 32 bits,
or, where `own` is true, through this package's entry points.  `exact` computes them from their definitions in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-5
BLOCK = 128
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1, "i8": 1}
QMAX = {"e4m3": 448.0, "i8": 127.0}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # decoding 16 sequences: bound by one read of both weights
        {"name": "gated 16x8192x4096 bf16", "op": "gated", "m": 16, "n": 8192, "k": 4096, "dtype": "bf16", "bias": False,
         "act": "silu", "save": False},
        # a training step's forward pass on the square shape of this repository's benchmark: pre-activations are kept
        {"name": "gated 4096x4096x4096 bf16", "op": "gated", "m": 4096, "n": 4096, "k": 4096, "dtype": "bf16", "bias": True,
         "act": "gelu_tanh", "save": True},
        # training: a short ragged batch in 16-bit floats, and the square shape
        {"name": "gated bwd 1000x500x2048 f16", "op": "gated_bwd", "m": 1000, "n": 500, "k": 2048, "dtype": "f16", "bias": True,
         "act": "gelu"},
        {"name": "gated bwd 4096x4096x4096 bf16", "op": "gated_bwd", "m": 4096, "n": 4096, "k": 4096, "dtype": "bf16",
         "bias": False, "act": "silu"},
        # the norm before a layer while decoding one sequence: latency alone
        {"name": "layer norm 1x4096 bf16", "op": "norm", "rows": 1, "d": 4096, "dtype": "bf16", "out": "bf16", "res": True,
         "bias": True},
        # a long prompt, the residual stream in 16 bits
        {"name": "layer norm 8192x8192 bf16", "op": "norm", "rows": 8192, "d": 8192, "dtype": "bf16", "out": "bf16", "res": True,
         "bias": True},
        # training in 32 bits with rows of an odd width, ragged; and a micro-batch of 8192 tokens in 16 bits
        {"name": "layer norm bwd 1000x2049 f32", "op": "norm_bwd", "rows": 1000, "d": 2049, "dtype": "f32", "res": False,
         "bias": False},
        {"name": "layer norm bwd 8192x4096 bf16", "op": "norm_bwd", "rows": 8192, "d": 4096, "dtype": "bf16", "res": True,
         "bias": True},
        # a ragged batch of gradients, transposed for the product that sums over its rows
        {"name": "blocks 1000x2000 f16 transposed", "op": "quant", "rows": 1000, "d": 2000, "dtype": "f16", "tall": False,
         "transpose": True},
        # the activations of a long prompt
        {"name": "blocks 8192x8192 bf16", "op": "quant", "rows": 8192, "d": 8192, "dtype": "bf16", "tall": False,
         "transpose": False},
        # decoding 16 sequences in 8 bits: bound by one read of the weight
        {"name": "block linear 16x8192x8192", "op": "block", "m": 16, "n": 8192, "k": 8192, "out": "bf16", "tall": True,
         "bias": False, "act": "none", "res": True},
        # a prompt of 4096 tokens in 8 bits
        {"name": "block linear 4096x4096x4096", "op": "block", "m": 4096, "n": 4096, "k": 4096, "out": "bf16", "tall": True,
         "bias": True, "act": "silu", "res": False},
    ]


def _size(rng, lo, hi, multiple=1):
    """A size whose logarithm is spread evenly over [lo, hi], rounded down to a multiple."""
    return max(multiple, int(math.exp(rng.uniform(math.log(lo), math.log(hi)))) // multiple * multiple)


def draw(rng):
    op = rng.choice(("gated", "gated", "gated_bwd", "norm", "norm_bwd", "quant", "block", "block"))
    if op in ("norm", "norm_bwd"):
        d = _size(rng, 64, 16384, rng.choice((1, 8, 64)))
        dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
        rows = _size(rng, 1, min(16384, (8192 * 8192 if op == "norm" else 8192 * 4096) // (d * SIZE[dtype] // 2)))
        case = {"op": op, "rows": rows, "d": d, "dtype": dtype, "res": rng.random() < 0.7, "bias": rng.random() < 0.8}
        if op == "norm":
            case["out"] = rng.choice((dtype, "e4m3"))
        return case
    if op == "quant":
        d = _size(rng, 64, 16384, rng.choice((1, 16, 128)))
        return {"op": op, "rows": _size(rng, 1, min(16384, 4096 * 8192 // d)), "d": d, "dtype": rng.choice(("bf16", "bf16", "f16", "f32")),
                "tall": rng.random() < 0.3, "transpose": rng.random() < 0.5}
    if op == "block":
        n, k = _size(rng, 64, 8192, rng.choice((1, 8, 128))), _size(rng, 64, 8192, rng.choice((16, 128)))
        m = _size(rng, 1, min(8192, 4096 ** 3 // (n * k)))
        return {"op": op, "m": m, "n": n, "k": k, "out": rng.choice(("bf16", "f16", "f32")), "tall": rng.random() < 0.7,
                "bias": rng.random() < 0.5, "act": rng.choice(ACTS), "res": rng.random() < 0.5}
    dtype = rng.choice(("bf16", "bf16", "f16", "e4m3", "i8")) if op == "gated" else rng.choice(("bf16", "bf16", "f16"))
    multiple = 16 if SIZE[dtype] == 1 else rng.choice((1, 8, 64)) if op == "gated" else rng.choice((8, 64))
    n, k = _size(rng, 64, 8192, multiple), _size(rng, 64, 8192, multiple)
    m = _size(rng, 1, min(8192, 4096 ** 3 // (n * k)))
    case = {"op": op, "m": m, "n": n, "k": k, "dtype": dtype, "bias": rng.random() < 0.5, "act": rng.choice(ACTS)}
    if op == "gated":
        case["save"] = rng.random() < 0.3
    return case


# ------------------------------------------------------------------ the inputs

def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * std


def _hidden(g, rows, d):
    """Rows as a network's hidden states are: normal entries whose size varies from channel to channel and from token to
    token, with a few channels far above the rest."""
    channel = torch.exp(_normal(g, d, std=0.4))
    channel[torch.randint(0, d, (max(1, d // 512),), generator=g, device="cuda")] *= 12.0
    return _normal(g, rows, d) * channel * torch.exp(_normal(g, rows, 1, std=0.3))


def _row_codes(w, q):
    """8-bit rows and their scales, as a serving program keeps them."""
    scale = (w.abs().amax(1) / QMAX[q]).clamp_min(2.0 ** -100)
    v = w / scale[:, None]
    return (v.round().to(torch.int8) if q == "i8" else v.to(DT[q])), scale


def _strided(scale):
    """The scales (rows, blocks) as the quantisation leaves them: consecutive rows next to each other in memory."""
    return scale.t().contiguous().t()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op in ("norm", "norm_bwd"):
        rows, d, dt = case["rows"], case["d"], DT[case["dtype"]]
        s["w"] = (1.0 + _normal(g, d, std=0.2)).to(dt)
        if op == "norm":
            s["b"] = _normal(g, d, std=0.2).to(dt) if case["bias"] else None
            s["x"] = (_hidden(g, rows, d) + 0.3).to(dt)
            s["r"] = _hidden(g, rows, d).mul_(2.0).to(dt) if case["res"] else None
        else:
            h = (_hidden(g, rows, d).mul_(2.0) + 0.3).to(dt)
            s["h"] = h
            s["mean"] = h.float().mean(1)
            s["rstd"] = ((h.float() - s["mean"][:, None]).square().mean(1) + EPS).rsqrt()
            s["dy"] = _normal(g, rows, d, std=0.02).to(dt)
            s["dh"] = _normal(g, rows, d, std=0.02).to(dt) if case["res"] else None
        return s
    if op == "quant":
        s["x"] = _hidden(g, case["rows"], case["d"]).to(DT[case["dtype"]])
        return s
    m, n, k = case["m"], case["n"], case["k"]
    if op == "block":
        s["x"], sx = _quantise(_hidden(g, m, k), False)
        s["w"], sw = _quantise(_normal(g, n, k, std=k ** -0.5), case["tall"])
        s["xs"], s["ws"] = _strided(sx), _strided(sw)
        s["b"] = _normal(g, n, std=0.2).to(torch.bfloat16) if case["bias"] else None
        s["r"] = _normal(g, m, n).to(DT[case["out"]]) if case["res"] else None
        return s
    dt = DT[case["dtype"]]
    w = _normal(g, 2 * n, k, std=k ** -0.5)
    wide = torch.bfloat16 if SIZE[case["dtype"]] == 1 else dt
    s["b"] = _normal(g, 2 * n, std=0.2).to(wide) if case["bias"] else None
    if SIZE[case["dtype"]] == 1:
        s["w"], s["ws"] = _row_codes(w, case["dtype"])
        s["x"], s["xs"] = _row_codes(_hidden(g, m, k), case["dtype"])
    else:
        s["w"], s["x"] = w.to(dt), _normal(g, m, k).to(dt)
    if op == "gated_bwd":
        s["z"] = _normal(g, m, 2 * n).to(dt)
        s["dy"] = _normal(g, m, n, std=0.1).to(dt)
    return s


# ------------------------------------------------------------------ the plain form

def _act(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0.0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2.0 * math.pi) ** -0.5
    if act == "gelu_tanh":
        c = (2.0 / math.pi) ** 0.5
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    return torch.ones_like(z)


def _padded(v, rows, cols):
    out = v.new_zeros(rows, cols)
    out[:v.shape[0], :v.shape[1]] = v
    return out


def _blocks(v, tall):
    """v padded with zeros to whole blocks, as (row blocks, rows of a block, column blocks, BLOCK)."""
    high = BLOCK if tall else 1
    rows, cols = -(-v.shape[0] // high) * high, -(-v.shape[1] // BLOCK) * BLOCK
    return _padded(v, rows, cols).reshape(rows // high, high, cols // BLOCK, BLOCK)


def _quantise(v, tall):
    """v in E4M3, and one scale per block."""
    t = _blocks(v, tall)
    scale = (t.abs().amax((1, 3)) / QMAX["e4m3"]).clamp_min(2.0 ** -100)
    q = (t * (1.0 / scale)[:, None, :, None]).reshape(t.shape[0] * t.shape[1], -1)
    return q[:v.shape[0], :v.shape[1]].contiguous().to(DT["e4m3"]), scale


def _spread(scale, rows, cols, tall):
    """A scale per element from one per block."""
    if tall:
        scale = scale.repeat_interleave(BLOCK, 0)[:rows]
    return scale.repeat_interleave(BLOCK, 1)[:, :cols]


def _plain_norm(s):
    h = s["x"].float()
    if s["r"] is not None:
        h = h + s["r"].float()
    mean = h.mean(1, keepdim=True)
    off = h - mean
    rstd = torch.rsqrt(off.square().mean(1, keepdim=True) + EPS)
    y = off * rstd * s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    out = {"h": h.to(DT[s["dtype"]])} if s["r"] is not None else {}
    if s["out"] == "e4m3":
        scale = (y.abs().amax(1) / QMAX["e4m3"]).clamp_min(2.0 ** -100)
        out["q"], out["scale"] = (y * (1.0 / scale)[:, None]).to(DT["e4m3"]), scale
    else:
        out["y"], out["mean"], out["rstd"] = y.to(DT[s["out"]]), mean[:, 0], rstd[:, 0]
    return out


def _plain_norm_bwd(s):
    dt = DT[s["dtype"]]
    xhat = (s["h"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["w"].float()
    dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    out = {"dx": dx.to(dt), "dw": (dy * xhat).sum(0).to(dt)}
    if s["bias"]:
        out["db"] = dy.sum(0).to(dt)
    return out


def _plain_quant(s):
    v = s["x"].float()
    q, scale = _quantise(v.t() if s["transpose"] else v, s["tall"])
    # codes of a transposed matrix end in zeros, up to whole chunks of 16
    return {"q": _padded(q.float(), q.shape[0], -(-q.shape[1] // 16) * 16).to(q.dtype) if s["transpose"] else q, "scale": scale}


def _plain_block(s):
    m, n, k = s["m"], s["n"], s["k"]
    z = (s["x"].float() * _spread(s["xs"], m, k, False)) @ (s["w"].float() * _spread(s["ws"], n, k, s["tall"])).t()
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(z, s["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    return {"y": y.to(DT[s["out"]])}


def _plain_gated(s):
    wide = torch.bfloat16 if SIZE[s["dtype"]] == 1 else DT[s["dtype"]]
    z = s["x"].float() @ s["w"].float().t()
    if SIZE[s["dtype"]] == 1:
        z = z * s["xs"][:, None] * s["ws"]
    if s["b"] is not None:
        z = z + s["b"].float()
    out = {"y": (_act(z[:, :s["n"]], s["act"]) * z[:, s["n"]:]).to(wide)}
    if s["save"]:
        out["z"] = z.to(wide)
    return out


def _plain_gated_bwd(s):
    dt, n = DT[s["dtype"]], s["n"]
    dy, gate, up = s["dy"].float(), s["z"][:, :n].float(), s["z"][:, n:].float()
    dz = torch.cat((dy * up * _act_slope(gate, s["act"]), dy * _act(gate, s["act"])), 1)
    out = {"dx": (dz @ s["w"].float()).to(dt), "dw": (dz.t() @ s["x"].float()).to(dt)}
    if s["b"] is not None:
        out["db"] = dz.sum(0).to(dt)
    return out


PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "quant": _plain_quant, "block": _plain_block, "gated": _plain_gated,
         "gated_bwd": _plain_gated_bwd}


# ------------------------------------------------------------------ this package's operators

def _own_norm(gb, s):
    if s["out"] == "e4m3":
        t = gb.add_layer_norm(s["x"], s["w"], s["b"], residual=s["r"], eps=EPS, out_dtype=torch.float8_e4m3fn)
        out = {"q": t.y, "scale": t.scale}
    else:
        t = gb.add_layer_norm(s["x"], s["w"], s["b"], residual=s["r"], eps=EPS, save_stats=True)
        out = {"y": t.y, "mean": t.mean, "rstd": t.rstd}
    if s["r"] is not None:
        out["h"] = t.h
    return out


def _own_norm_bwd(gb, s):
    t = gb.add_layer_norm_backward(s["dy"], s["h"], s["w"], s["mean"], s["rstd"], dh=s["dh"], bias_grad=s["bias"])
    out = {"dx": t.dx, "dw": t.dweight}
    if s["bias"]:
        out["db"] = t.dbias
    return out


def _own_quant(gb, s):
    t = gb.quantize_blocks(s["x"], block=(BLOCK, BLOCK) if s["tall"] else (1, BLOCK), transpose=s["transpose"])
    return {"q": t.q, "scale": t.scale}


def _own_block(gb, s):
    return {"y": gb.block_linear(s["x"], s["w"], s["xs"], s["ws"], bias=s["b"], activation=s["act"], residual=s["r"],
                                 out_dtype=DT[s["out"]])}


def _own_gated(gb, s):
    t = gb.gated_linear(s["x"], s["w"], bias=s["b"], activation=s["act"], x_scale=s.get("xs"), weight_scale=s.get("ws"),
                        save_preact=s["save"])
    return {"y": t[0], "z": t[1]} if s["save"] else {"y": t}


def _own_gated_bwd(gb, s):
    t = gb.gated_linear_backward(s["dy"], s["x"], s["w"], s["z"], activation=s["act"], bias_grad=s["b"] is not None)
    out = {"dx": t.dx, "dw": t.dweight}
    if s["b"] is not None:
        out["db"] = t.dbias
    return out


OWN = {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "quant": _own_quant, "block": _own_block, "gated": _own_gated,
       "gated_bwd": _own_gated_bwd}


def run(state):
    if own:
        import dense_tiled_gemm_amd as gb

        return OWN[state["op"]](gb, state)
    return PLAIN[state["op"]](state)


# ------------------------------------------------------------------ bytes and operations

def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        e, cells, d = SIZE[case["dtype"]], case["rows"] * case["d"], case["d"]
        if op == "norm_bwd":  # dy, h and dx, with the residual dh; w, dw and db; mean and rstd
            return {"bytes": cells * e * (4 if case["res"] else 3) + (2 + case["bias"]) * d * e + 8 * case["rows"], "flops": 12 * cells}
        # x and y, with the residual r and h; w and b; mean and rstd, or the scales
        return {"bytes": cells * (e * (3 if case["res"] else 1) + SIZE[case["out"]]) + (1 + case["bias"]) * d * e
                + case["rows"] * (4 if case["out"] == "e4m3" else 8), "flops": 8 * cells}
    if op == "quant":
        rows, cols = (case["d"], case["rows"]) if case["transpose"] else (case["rows"], case["d"])
        scales = -(-rows // (BLOCK if case["tall"] else 1)) * -(-cols // BLOCK)
        return {"bytes": rows * cols * (SIZE[case["dtype"]] + 1) + 4 * scales, "flops": 3 * rows * cols}
    m, n, k = case["m"], case["n"], case["k"]
    if op == "block":
        scales = (m + -(-n // (BLOCK if case["tall"] else 1))) * -(-k // BLOCK)
        return {"bytes": m * k + n * k + 4 * scales + 2 * n * case["bias"] + m * n * SIZE[case["out"]] * (1 + case["res"]),
                "flops": 2 * m * n * k}
    e = SIZE[case["dtype"]]
    if op == "gated_bwd":  # dy, z, x, w and dx, dw, db
        return {"bytes": (3 * m * n + 2 * m * k + 4 * n * k + 2 * n * case["bias"]) * e, "flops": 8 * m * n * k}
    scales = 4 * (m + 2 * n) if e == 1 else 0
    return {"bytes": (m * k + 2 * n * k) * e + scales + 2 * (2 * n * case["bias"] + m * n * (3 if case["save"] else 1)),
            "flops": 4 * m * n * k}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_act(z, act):
    """act(z) and its derivative."""
    one = torch.ones_like(z)
    if act == "none":
        return z, one
    if act == "relu":
        return torch.where(z > 0, z, 0 * one), torch.where(z > 0, one, 0 * one)
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    if act == "gelu":  # z times the normal distribution's function, whose derivative is its density
        p = torch.special.ndtr(z)
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    u = math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)  # (1 + tanh(u/2)) / 2 = sigmoid(u)
    p = torch.sigmoid(u)
    return z * p, p + z * p * (1 - p) * math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * z ** 2)


def _exact_codes(u):
    """u rounded to E4M3: 3 bits after the leading one, the smallest exponent -6."""
    step = torch.exp2(torch.floor(torch.log2(u.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(u / step) * step


def _index(n, high, device):
    """The block that each of n rows or columns lies in."""
    return torch.arange(n, device=device) // high


def exact(case, seed):
    s = prepare(case, seed)
    f = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    op = case["op"]
    if op == "norm":
        h = f["x"] + f["r"] if "r" in f else f["x"]
        mean = h.sum(1) / case["d"]
        std = torch.sqrt(((h - mean[:, None]) ** 2).sum(1) / case["d"] + EPS)
        y = (h - mean[:, None]) / std[:, None] * f["w"] + f.get("b", 0)
        out = {"h": h} if "r" in f else {}
        if case["out"] == "e4m3":
            scale = torch.clamp(y.abs().max(1).values / 448, min=2.0 ** -100)
            out["q"], out["scale"] = _exact_codes(y / scale[:, None]), scale
        else:
            out.update(y=y, mean=mean, rstd=1 / std)
        return out
    if op == "norm_bwd":
        d, r = case["d"], f["rstd"][:, None]
        off = f["h"] - f["mean"][:, None]
        g = f["dy"] * f["w"]
        dx = r * g - r / d * g.sum(1, keepdim=True) - r ** 3 / d * off * (g * off).sum(1, keepdim=True) + f.get("dh", 0)
        out = {"dx": dx, "dw": (f["dy"] * off * r).sum(0)}
        if case["bias"]:
            out["db"] = f["dy"].sum(0)
        return out
    if op == "quant":
        v = f["x"].t() if case["transpose"] else f["x"]
        rows, cols = v.shape
        i = _index(rows, BLOCK if case["tall"] else 1, v.device)
        j = _index(cols, BLOCK, v.device)
        top = v.new_zeros(rows, int(j[-1]) + 1).scatter_reduce(1, j.expand(rows, cols), v.abs(), "amax")
        top = v.new_zeros(int(i[-1]) + 1, top.shape[1]).scatter_reduce(0, i[:, None].expand_as(top), top, "amax")
        scale = torch.clamp(top / 448, min=2.0 ** -100)
        q = _exact_codes(v / scale[i][:, j])
        if case["transpose"] and cols % 16:
            q = torch.cat((q, q.new_zeros(rows, 16 - cols % 16)), 1)
        return {"q": q, "scale": scale}
    if op == "block":
        j = _index(case["k"], BLOCK, s["x"].device)
        w = f["w"] * f["ws"][_index(case["n"], BLOCK if case["tall"] else 1, j.device)][:, j]
        y = torch.mm(f["x"] * f["xs"][:, j], w.t().contiguous()) + f.get("b", 0)
        return {"y": _exact_act(y, case["act"])[0] + f.get("r", 0)}
    n = case["n"]
    if op == "gated_bwd":
        value, slope = _exact_act(f["z"][:, :n].contiguous(), case["act"])
        dz = f["dy"].new_empty(case["m"], 2 * n)
        dz[:, :n], dz[:, n:] = f["dy"] * f["z"][:, n:] * slope, f["dy"] * value
        out = {"dx": torch.mm(dz, f["w"]), "dw": torch.mm(dz.t().contiguous(), f["x"])}
        if "b" in f:
            out["db"] = dz.sum(0)
        return out
    x, w = (f["x"] * f["xs"][:, None], f["w"] * f["ws"][:, None]) if "xs" in f else (f["x"], f["w"])
    z = torch.mm(x, w.t().contiguous()) + f.get("b", 0)
    out = {"y": _exact_act(z[:, :n].contiguous(), case["act"])[0] * z[:, n:]}
    if case["save"]:
        out["z"] = z
    return out
