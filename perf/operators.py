"""The operators around the matrix product: what they compute in plain form, and the cases they are measured on.

The operators are those of a pre-norm block of a language model: the root-mean-square norm with the residual's
addition (out in 16 or 32 bits, or in 8 bits with one scale per row), the matrix product with bias, activation and
residual in its epilogue, the product of 8-bit rows with their scales, and the backward passes of the norm and of the
product.  `run` computes them with elementary torch operations in 32 bits, or, where `own` is true, through this
package's entry points.  `exact` computes them from their definitions in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1, "i8": 1}
QMAX = {"e4m3": 448.0, "i8": 127.0}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the norm before a layer while decoding one sequence: latency alone
        {"name": "norm 1x4096 bf16", "op": "norm", "rows": 1, "d": 4096, "dtype": "bf16", "out": "bf16", "res": True},
        # an odd width and a ragged number of tokens, rows that are only 2-byte aligned; the first norm has no residual
        {"name": "norm 1000x2049 f16", "op": "norm", "rows": 1000, "d": 2049, "dtype": "f16", "out": "f16", "res": False},
        # a long prompt in front of an 8-bit product: the norm leaves E4M3 rows with their scales
        {"name": "norm 8192x8192 bf16-e4m3", "op": "norm", "rows": 8192, "d": 8192, "dtype": "bf16", "out": "e4m3", "res": True},
        # training, a micro-batch of 8192 tokens
        {"name": "norm bwd 8192x4096 bf16", "op": "norm_bwd", "rows": 8192, "d": 4096, "dtype": "bf16", "res": True},
        # training in 32 bits, ragged
        {"name": "norm bwd 1000x2050 f32", "op": "norm_bwd", "rows": 1000, "d": 2050, "dtype": "f32", "res": False},
        # decoding 16 sequences: bound by one read of the weight
        {"name": "linear 16x8192x8192 bf16", "op": "linear", "m": 16, "n": 8192, "k": 8192, "dtype": "bf16", "out": "bf16",
         "bias": True, "act": "silu", "res": False, "save": False},
        # the ragged shape of this repository's benchmark, f32 results with a residual
        {"name": "linear 1000x3000x2050 f16", "op": "linear", "m": 1000, "n": 3000, "k": 2050, "dtype": "f16", "out": "f32",
         "bias": True, "act": "gelu", "res": True, "save": False},
        # the square shape of this repository's benchmark as a training step's forward pass: the pre-activation is kept
        {"name": "linear 4096x4096x4096 bf16", "op": "linear", "m": 4096, "n": 4096, "k": 4096, "dtype": "bf16", "out": "bf16",
         "bias": True, "act": "gelu_tanh", "res": True, "save": True},
        # serving in int8, 64 sequences: 16-bit rows are quantised, then multiplied
        {"name": "qlinear 64x8192x8192 i8", "op": "qlinear", "m": 64, "n": 8192, "k": 8192, "dtype": "bf16", "q": "i8",
         "bias": False, "act": "none", "res": True},
        # serving a prompt of 4096 tokens in E4M3
        {"name": "qlinear 4096x4096x4096 e4m3", "op": "qlinear", "m": 4096, "n": 4096, "k": 4096, "dtype": "bf16", "q": "e4m3",
         "bias": True, "act": "silu", "res": False},
        # training: a short ragged batch, and the square shape
        {"name": "linear bwd 1000x512x2048 f16", "op": "linear_bwd", "m": 1000, "n": 512, "k": 2048, "dtype": "f16",
         "bias": True, "act": "relu"},
        {"name": "linear bwd 4096x4096x4096 bf16", "op": "linear_bwd", "m": 4096, "n": 4096, "k": 4096, "dtype": "bf16",
         "bias": True, "act": "gelu_tanh"},
    ]


def _size(rng, lo, hi, multiple=1):
    """A size whose logarithm is spread evenly over [lo, hi], rounded down to a multiple."""
    size = max(multiple, int(math.exp(rng.uniform(math.log(lo), math.log(hi)))) // multiple * multiple)
    return size if size != 3072 else size - multiple


def draw(rng):
    op = rng.choice(("norm", "norm_bwd", "linear", "qlinear", "linear_bwd"))
    if op in ("norm", "norm_bwd"):
        d = _size(rng, 64, 16384, rng.choice((1, 8, 64)))
        rows = _size(rng, 1, min(16384, (8192 * 8192 if op == "norm" else 8192 * 4096) // d))
        dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
        case = {"op": op, "rows": rows, "d": d, "dtype": dtype, "res": rng.random() < 0.7}
        if dtype == "f32":
            case["rows"] = max(1, rows // 2)
        if op == "norm":
            case["out"] = rng.choice((dtype, "e4m3"))
        return case
    multiple = {"linear": rng.choice((1, 8, 64)), "qlinear": 16, "linear_bwd": rng.choice((8, 64))}[op]
    n, k = _size(rng, 64, 8192, multiple), _size(rng, 64, 8192, multiple)
    m = _size(rng, 1, min(8192, 4096 ** 3 // (n * k)))
    case = {"op": op, "m": m, "n": n, "k": k, "dtype": rng.choice(("bf16", "bf16", "f16")), "bias": rng.random() < 0.7,
            "act": rng.choice(ACTS)}
    if op == "linear":
        case.update(out=rng.choice((case["dtype"], "f32")), res=rng.random() < 0.5, save=rng.random() < 0.3)
    if op == "qlinear":
        case.update(q=rng.choice(("e4m3", "i8")), res=rng.random() < 0.5)
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


def _quantised_weight(w, q):
    """8-bit rows of a weight and their scales, as a serving program keeps them."""
    scale = w.abs().amax(1) / QMAX[q]
    v = w / scale[:, None]
    return (v.round().to(torch.int8) if q == "i8" else v.to(DT[q])), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dt = case["op"], DT[case["dtype"]]
    s = dict(case)
    if op in ("norm", "norm_bwd"):
        rows, d = case["rows"], case["d"]
        s["w"] = (1.0 + _normal(g, d, std=0.2)).to(dt)
        if op == "norm":
            s["x"] = _hidden(g, rows, d).to(dt)
            s["r"] = _hidden(g, rows, d).mul_(2.0).to(dt) if case["res"] else None
        else:
            h = _hidden(g, rows, d).mul_(2.0).to(dt)
            s["h"] = h
            s["rstd"] = (h.float().square().mean(1) + EPS).rsqrt()
            s["dy"] = _normal(g, rows, d, std=0.02).to(dt)
            s["dh"] = _normal(g, rows, d, std=0.02).to(dt) if case["res"] else None
        return s
    m, n, k = case["m"], case["n"], case["k"]
    w = _normal(g, n, k, std=k ** -0.5)
    s["b"] = _normal(g, n, std=0.2).to(dt) if case["bias"] else None
    if op == "linear_bwd":
        s["w"] = w.to(dt)
        s["x"] = _normal(g, m, k).to(dt)
        s["z"] = _normal(g, m, n).to(dt) if case["act"] != "none" else None
        s["dy"] = _normal(g, m, n, std=0.1).to(dt)
        return s
    if op == "qlinear":
        s["w"], s["ws"] = _quantised_weight(w, case["q"])
        s["x"] = _hidden(g, m, k).to(dt)
    else:
        s["w"] = w.to(dt)
        s["x"] = _normal(g, m, k).to(dt)
    s["r"] = _normal(g, m, n).to(DT[case.get("out", case["dtype"])]) if case["res"] else None
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


def _quantise(v, q):
    """Rows of v in 8 bits, and one scale per row."""
    scale = (v.abs().amax(1) / QMAX[q]).clamp_min(2.0 ** -100)
    u = v * (1.0 / scale)[:, None]
    return (torch.round(u).to(torch.int8) if q == "i8" else u.to(DT[q])), scale


def _plain_norm(s):
    h = s["x"].float()
    if s["r"] is not None:
        h = h + s["r"].float()
    rstd = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
    y = h * rstd * s["w"].float()
    out = {"h": h.to(DT[s["dtype"]])} if s["r"] is not None else {}
    if s["out"] == "e4m3":
        out["q"], out["scale"] = _quantise(y, "e4m3")
    else:
        out["y"], out["rstd"] = y.to(DT[s["out"]]), rstd[:, 0]
    return out


def _plain_norm_bwd(s):
    xhat = s["h"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["w"].float()
    dx = s["rstd"][:, None] * (g - xhat * (g * xhat).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(DT[s["dtype"]]), "dw": (dy * xhat).sum(0).to(DT[s["dtype"]])}


def _plain_product(s, x, w, out):
    z = x @ w.t()
    if s["op"] == "qlinear":
        z = z * s["xs"][:, None] * s["ws"]
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(z, s["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    got = {"y": y.to(out)}
    if s.get("save"):
        got["z"] = z.to(DT[s["dtype"]])
    return got


def _plain_linear(s):
    return _plain_product(s, s["x"].float(), s["w"].float(), DT[s["out"]])


def _plain_qlinear(s):
    q, scale = _quantise(s["x"].float(), s["q"])
    return _plain_product({**s, "xs": scale}, q.float(), s["w"].float(), DT[s["dtype"]])


def _plain_linear_bwd(s):
    dt = DT[s["dtype"]]
    dz = s["dy"].float()
    if s["act"] != "none":
        dz = dz * _act_slope(s["z"].float(), s["act"])
    out = {"dx": (dz @ s["w"].float()).to(dt), "dw": (dz.t() @ s["x"].float()).to(dt)}
    if s["b"] is not None:
        out["db"] = dz.sum(0).to(dt)
    return out


PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "linear": _plain_linear, "qlinear": _plain_qlinear,
         "linear_bwd": _plain_linear_bwd}


# ------------------------------------------------------------------ this package's operators

def _own_norm(gb, s):
    if s["out"] == "e4m3":
        t = gb.add_rms_norm(s["x"], s["w"], residual=s["r"], eps=EPS, out_dtype=torch.float8_e4m3fn)
        out = {"q": t.y, "scale": t.scale}
    else:
        t = gb.add_rms_norm(s["x"], s["w"], residual=s["r"], eps=EPS, save_rstd=True)
        out = {"y": t.y, "rstd": t.rstd}
    if s["r"] is not None:
        out["h"] = t.h
    return out


def _own_norm_bwd(gb, s):
    dx, dw = gb.add_rms_norm_backward(s["dy"], s["h"], s["w"], s["rstd"], dh=s["dh"])
    return {"dx": dx, "dw": dw}


def _own_linear(gb, s):
    t = gb.linear(s["x"], s["w"], bias=s["b"], activation=s["act"], residual=s["r"], out_dtype=DT[s["out"]],
                  save_preact=s["save"])
    return {"y": t[0], "z": t[1]} if s["save"] else {"y": t}


def _own_qlinear(gb, s):
    q, scale = gb.quantize_rows(s["x"], DT[s["q"]])
    return {"y": gb.linear(q, s["w"], bias=s["b"], activation=s["act"], residual=s["r"], x_scale=scale, weight_scale=s["ws"],
                           out_dtype=DT[s["dtype"]])}


def _own_linear_bwd(gb, s):
    t = gb.linear_backward(s["dy"], s["x"], s["w"], preact=s["z"], activation=s["act"], bias_grad=s["b"] is not None)
    out = {"dx": t.dx, "dw": t.dweight}
    if s["b"] is not None:
        out["db"] = t.dbias
    return out


OWN = {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "linear": _own_linear, "qlinear": _own_qlinear,
       "linear_bwd": _own_linear_bwd}


def run(state):
    if own:
        import dense_tiled_gemm_amd as gb

        return OWN[state["op"]](gb, state)
    return PLAIN[state["op"]](state)


# ------------------------------------------------------------------ bytes and operations

def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    if op in ("norm", "norm_bwd"):
        cells, d = case["rows"] * case["d"], case["d"]
        if op == "norm_bwd":  # dy, h and dx, with the residual dh; w and dw; rstd
            return {"bytes": cells * e * (4 if case["res"] else 3) + 2 * d * e + 4 * case["rows"], "flops": 10 * cells}
        # x and y, with the residual r and h; w; rstd or the scales
        return {"bytes": cells * (e * (3 if case["res"] else 1) + SIZE[case["out"]]) + d * e + 4 * case["rows"], "flops": 6 * cells}
    m, n, k = case["m"], case["n"], case["k"]
    if op == "linear_bwd":  # dy, z, x, w and dx, dw, db
        size = m * n * (1 if case["act"] == "none" else 2) + 2 * m * k + 2 * n * k + n * case["bias"]
        return {"bytes": size * e, "flops": 4 * m * n * k}
    if op == "qlinear":
        return {"bytes": m * k * e + n * k + 4 * n + (n * case["bias"] + m * n * (1 + case["res"])) * e, "flops": 2 * m * n * k}
    o = SIZE[case["out"]]
    size = (m * k + n * k + n * case["bias"] + m * n * case["save"]) * e + m * n * o * (1 + case["res"])
    return {"bytes": size, "flops": 2 * m * n * k}


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


def _exact_codes(v, q):
    """The values of v's rows in 8 bits (in units of their scales), and the scales."""
    scale = torch.clamp(v.abs().max(1).values / QMAX[q], min=2.0 ** -100)
    u = v / scale[:, None]
    if q == "i8":
        return torch.round(u), scale
    # E4M3: 3 bits after the leading one, the smallest exponent -6
    step = torch.exp2(torch.floor(torch.log2(u.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(u / step) * step, scale


def exact(case, seed):
    s = prepare(case, seed)
    f = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    op = case["op"]
    if op == "norm":
        h = f["x"] + f["r"] if "r" in f else f["x"]
        rms = torch.sqrt((h * h).sum(1) / case["d"] + EPS)
        y = h / rms[:, None] * f["w"]
        out = {"h": h} if "r" in f else {}
        if case["out"] == "e4m3":
            out["q"], out["scale"] = _exact_codes(y, "e4m3")
        else:
            out.update(y=y, rstd=1 / rms)
        return out
    if op == "norm_bwd":
        rstd = f["rstd"][:, None]
        g = f["dy"] * f["w"]
        dx = rstd * g - rstd ** 3 * f["h"] * (g * f["h"]).sum(1, keepdim=True) / case["d"] + f.get("dh", 0)
        return {"dx": dx, "dw": (f["dy"] * f["h"] * rstd).sum(0)}
    if op == "linear_bwd":
        dz = f["dy"] if case["act"] == "none" else f["dy"] * _exact_act(f["z"], case["act"])[1]
        out = {"dx": torch.mm(dz, f["w"]), "dw": torch.mm(dz.t().contiguous(), f["x"])}
        if "b" in f:
            out["db"] = dz.sum(0)
        return out
    if op == "qlinear":
        q, scale = _exact_codes(f["x"], case["q"])
        z = torch.mm(q * scale[:, None], (f["w"] * f["ws"][:, None]).t().contiguous())
    else:
        z = torch.mm(f["x"], f["w"].t().contiguous())
    if "b" in f:
        z = z + f["b"]
    y = _exact_act(z, case["act"])[0]
    out = {"y": y + f["r"] if "r" in f else y}
    if case.get("save"):
        out["z"] = z
    return out
