"""The microscaled (MX) operators: what is measured, and their plain forms.

Formats: blocks of 32 consecutive values of a row share one power of two
2^(s - 127), held as the byte s (255 = NaN).  MXFP4 holds values as e2m1 (0,
0.5, 1, 1.5, 2, 3, 4, 6 and a sign bit), two to a byte, the even position in
the low nibble; MXFP8 as e4m3 bytes.  A block's exponent is that of its
largest magnitude less 2 (e2m1) or 8 (e4m3), at least -127; values are divided
by it, rounded to nearest even and held at the largest value (6 or 448).

  quantize  rows to codes and scales (MXFP4: and back, as a weight is checked
            or a straight-through training step uses it)
  rmsnorm   r' = x + r; h = r' * rsqrt(mean(r'^2) + eps) * w; h as MXFP8
  matmul    Y[t, o] = sum_k A[t, k] W[o, k], W in MXFP4, A in MXFP8 or MXFP4
  moe       a mixture-of-experts layer: top-k of the router's logits, softmax
            over the chosen ones, each expert down(silu(gate x) * up x)
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-5
FP4_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decoding step's activations on their way into one product
        {"name": "quantize fp8 1x4096", "op": "quantize", "format": "fp8", "type": "bf16",
         "rows": 1, "dim": 4096},
        # a weight matrix quantised once and read back (4096 -> 14336)
        {"name": "quantize fp4 14336x4096", "op": "quantize", "format": "fp4", "type": "fp32",
         "rows": 14336, "dim": 4096},
        # ragged batch, odd number of blocks in a row
        {"name": "quantize fp4 333x1056", "op": "quantize", "format": "fp4", "type": "fp16",
         "rows": 333, "dim": 1056},
        # one token between two layers
        {"name": "rmsnorm 1x4096", "op": "rmsnorm", "type": "bf16", "rows": 1, "dim": 4096},
        # a prompt, between two layers
        {"name": "rmsnorm 4096x5120", "op": "rmsnorm", "type": "bf16", "rows": 4096, "dim": 5120},
        # single token: latency and the weight stream
        {"name": "matmul 1x4096x4096", "op": "matmul", "format": "fp8", "type": "fp32",
         "tokens": 1, "dim": 4096, "out": 4096},
        # a decoding batch through the FFN's up projection
        {"name": "matmul 64x4096x14336", "op": "matmul", "format": "fp8", "type": "bf16",
         "tokens": 64, "dim": 4096, "out": 14336},
        # odd sizes, both operands in 4 bits
        {"name": "matmul fp4 333x1056x4097", "op": "matmul", "format": "fp4", "type": "fp16",
         "tokens": 333, "dim": 1056, "out": 4097},
        # a long prompt through the FFN's up projection
        {"name": "matmul 4096x4096x14336", "op": "matmul", "format": "fp8", "type": "bf16",
         "tokens": 4096, "dim": 4096, "out": 14336},
        # one token, many small experts
        {"name": "moe 1 of 64 experts", "op": "moe", "type": "bf16", "tokens": 1, "dim": 2048,
         "ffn": 1024, "experts": 64, "top_k": 8},
        # a decoding batch, odd sizes, activations in 32 bits
        {"name": "moe 13 of 24 experts", "op": "moe", "type": "fp32", "tokens": 13, "dim": 1056,
         "ffn": 736, "experts": 24, "top_k": 3},
        # a decoding batch that reaches every one of a few large experts
        {"name": "moe 32 of 8 experts", "op": "moe", "type": "bf16", "tokens": 32, "dim": 4096,
         "ffn": 14336, "experts": 8, "top_k": 2},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _dim(rng, low, high):
    return 32 * max(1, _log(rng, low, high) // 32)


def draw(rng):
    op = rng.choice(["quantize", "rmsnorm", "matmul", "moe"])
    kind = rng.choice(["fp32", "bf16", "fp16"])
    if op in ("quantize", "rmsnorm"):
        dim = _dim(rng, 32, 16384)
        rows = min(_log(rng, 1, 8192), (1 << 25) // dim)
        case = {"op": op, "type": kind, "rows": rows, "dim": dim}
        if op == "quantize":
            case["format"] = rng.choice(["fp4", "fp8"])
        return case
    if op == "matmul":
        dim, out = _dim(rng, 32, 8192), _log(rng, 1, 8192)
        return {"op": op, "type": kind, "format": rng.choice(["fp4", "fp8"]),
                "tokens": min(_log(rng, 1, 4096), (1 << 37) // (dim * out)), "dim": dim, "out": out}
    experts, dim = _log(rng, 2, 64), _dim(rng, 64, 4096)
    ffn = min(_dim(rng, 32, 4096), 32 * ((1 << 23) // (experts * dim)))
    return {"op": op, "type": kind, "tokens": _log(rng, 1, 64), "dim": dim, "ffn": ffn,
            "experts": experts, "top_k": rng.randint(1, min(8, experts))}


def work(case):
    size = {"fp32": 4, "bf16": 2, "fp16": 2}[case["type"]]
    op, K = case["op"], case["dim"]
    code = {"fp4": 0.5, "fp8": 1.0}[case.get("format", "fp8")] + 1 / 32
    if op == "quantize":
        n = case["rows"] * K
        back = 2 if case["format"] == "fp4" else 0
        return {"bytes": n * (size + back + (0 if back else code)), "flops": 2 * n}
    if op == "rmsnorm":
        n = case["rows"] * K
        return {"bytes": n * (3 * size + code) + K * size, "flops": 6 * n}
    if op == "matmul":
        M, N = case["tokens"], case["out"]
        return {"bytes": M * K * code + N * K * (0.5 + 1 / 32) + M * N * size,
                "flops": 2 * M * N * K}
    M, F, E, k = case["tokens"], case["ffn"], case["experts"], case["top_k"]
    reached = E * (1 - (1 - k / E) ** M)  # experts that M even choices of k of E reach
    return {"bytes": reached * 3 * K * F * (0.5 + 1 / 32) + E * K * size + 2 * M * K * size,
            "flops": 2 * M * (k * 3 * K * F + E * K)}


# ---------------------------------------------------------------- inputs

def _rng(seed):
    g = torch.Generator(DEV)
    g.manual_seed(int(seed))
    return g


def _activations(g, rows, dim, dtype):
    """Normal values with a spread of channel sizes, a few of them large."""
    channel = torch.exp(0.6 * torch.randn(dim, generator=g, device=DEV))
    return (torch.randn(rows, dim, generator=g, device=DEV) * channel).to(dtype)


def prepare(case, seed):
    dtype, K = TYPES[case["type"]], case["dim"]
    s = dict(case)
    g = _rng(seed)

    def packed(rows, dim, fmt="fp4"):
        """Codes and scales of normal values, quantised some rows at a time."""
        codes = torch.empty(rows, dim // 2 if fmt == "fp4" else dim, dtype=torch.uint8, device=DEV)
        scales = torch.empty(rows, dim // 32, dtype=torch.uint8, device=DEV)
        step = max(1, (1 << 26) // dim)
        for a in range(0, rows, step):
            x = torch.randn(min(step, rows - a), dim, generator=g, device=DEV)
            if fmt == "fp8":
                x = x * torch.exp(0.6 * torch.randn(dim, generator=g, device=DEV))
            c, t = _quantize(x * (dim ** -0.5 if fmt == "fp4" else 1.0), fmt)
            codes[a:a + step] = _pack(c) if fmt == "fp4" else c.view(torch.uint8)
            scales[a:a + step] = t
        return codes, scales

    if case["op"] == "quantize":
        rows, fp4 = case["rows"], case["format"] == "fp4"
        s["x"] = _activations(g, rows, K, dtype)
        s["codes"] = torch.empty(rows, K // 2 if fp4 else K, dtype=torch.uint8, device=DEV)
        s["scales"] = torch.empty(rows, K // 32, dtype=torch.uint8, device=DEV)
        s["y"] = torch.empty(rows, K, dtype=torch.bfloat16, device=DEV) if fp4 else None
    elif case["op"] == "rmsnorm":
        rows = case["rows"]
        s["x"] = _activations(g, rows, K, dtype)
        s["residual"] = _activations(g, rows, K, dtype)
        s["weight"] = (1 + 0.2 * torch.randn(K, generator=g, device=DEV)).to(dtype)
        s["residual_out"] = torch.empty_like(s["x"])
        s["codes"] = torch.empty(rows, K, dtype=torch.uint8, device=DEV)
        s["scales"] = torch.empty(rows, K // 32, dtype=torch.uint8, device=DEV)
    elif case["op"] == "matmul":
        s["a_codes"], s["a_scales"] = packed(case["tokens"], K, case["format"])
        s["w_codes"], s["w_scales"] = packed(case["out"], K)
        s["y"] = torch.empty(case["tokens"], case["out"], dtype=dtype, device=DEV)
    else:
        E, F = case["experts"], case["ffn"]
        s["x"] = torch.randn(case["tokens"], K, generator=g, device=DEV).to(dtype)
        s["router"] = (1.5 * K ** -0.5 * torch.randn(E, K, generator=g, device=DEV)).to(dtype)
        s["bias"] = 0.3 * torch.randn(E, generator=g, device=DEV)
        c, t = packed(E * 2 * F, K)
        s["up_codes"], s["up_scales"] = c.view(E, 2 * F, -1), t.view(E, 2 * F, -1)
        c, t = packed(E * K, F)
        s["down_codes"], s["down_scales"] = c.view(E, K, -1), t.view(E, K, -1)
        s["y"] = torch.empty_like(s["x"])
    return s


# ---------------------------------------------------------------- plain forms

def _quantize(x, fmt):
    """(codes, scale bytes) of rows: e2m1 codes one to a byte, or e4m3 values."""
    b = x.float().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    e = torch.frexp(amax).exponent - 1 - (2 if fmt == "fp4" else 8)
    e = torch.where(amax > 0, e, -127).clamp(min=-127)
    v = torch.ldexp(b, -e.unsqueeze(-1)).flatten(-2)
    scales = (e + 127).to(torch.uint8)
    if fmt == "fp8":
        return v.clamp(-448, 448).to(torch.float8_e4m3fn), scales
    a = v.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5))
    return code + 8 * torch.signbit(v), scales


def _pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _power(scales):
    return torch.ldexp(torch.ones((), device=scales.device), scales.int() - 127)


def _values(codes, scales, fmt):
    """What codes and scales stand for, in 32 bits."""
    if fmt == "fp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        one = torch.tensor(FP4_VALUES + tuple(-x for x in FP4_VALUES), device=codes.device)
        pair = torch.stack([one.repeat(16), one.repeat_interleave(16)], -1)
        v = pair[codes.int()].flatten(-2)
    return (v.unflatten(-1, (-1, 32)) * _power(scales).unsqueeze(-1)).flatten(-2)


def _plain_quantize(s):
    codes, scales = _quantize(s["x"], s["format"])
    if s["format"] == "fp8":
        return {"values": codes, "scales": scales.view(torch.float8_e8m0fnu)}
    return {"values": _values(_pack(codes), scales, "fp4").to(torch.bfloat16)}


def _plain_rmsnorm(s):
    r = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    f = r.float()
    h = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    values, scales = _quantize(h, "fp8")
    return {"residual": r, "values": values, "scales": scales.view(torch.float8_e8m0fnu)}


def _plain_matmul(s):
    a = _values(s["a_codes"], s["a_scales"], s["format"])
    w = _values(s["w_codes"], s["w_scales"], "fp4")
    return {"y": torch.matmul(a, w.t()).to(s["y"].dtype)}


def _plain_moe(s):
    x, k, F = s["x"], s["top_k"], s["ffn"]
    # in 64 bits: a logit next to the border of the chosen ones decides
    logits = torch.matmul(x.double(), s["router"].double().t()) + s["bias"].double()
    top, chosen = torch.sort(logits, dim=-1, descending=True, stable=True)
    top, chosen = top[:, :k].float(), chosen[:, :k]
    p = torch.exp(top - top[:, :1])
    p = p / p.sum(-1, keepdim=True)
    x = x.float()
    if x.shape[0] * k <= s["experts"]:  # the chosen experts' weights, one by one
        at = chosen.flatten()
        up = _values(s["up_codes"][at], s["up_scales"][at], "fp4")
        down = _values(s["down_codes"][at], s["down_scales"][at], "fp4")
        gu = torch.matmul(up, x.repeat_interleave(k, 0).unsqueeze(-1)).squeeze(-1)
        h = gu[:, :F] / (1 + torch.exp(-gu[:, :F])) * gu[:, F:]
        y = torch.matmul(down, h.unsqueeze(-1)).squeeze(-1).unflatten(0, (-1, k))
        return {"y": (y * p.unsqueeze(-1)).sum(1).to(s["x"].dtype)}
    up = _values(s["up_codes"], s["up_scales"], "fp4")  # every expert for every token
    gu = torch.matmul(x, up.flatten(0, 1).t()).unflatten(-1, (-1, 2 * F))
    h = gu[..., :F] / (1 + torch.exp(-gu[..., :F])) * gu[..., F:]
    share = torch.zeros_like(logits, dtype=torch.float32).scatter(1, chosen, p)
    h = h * share.unsqueeze(-1)
    down = _values(s["down_codes"], s["down_scales"], "fp4")
    y = torch.matmul(h.flatten(1), down.transpose(1, 2).reshape(-1, x.shape[1]))
    return {"y": y.to(s["x"].dtype)}


# ---------------------------------------------------------------- the framework's calls

def _own_quantize(s):
    from q4_packed_weight_amd import binding
    binding.mx_quantize(s["x"], s["rows"], s["dim"], s["format"], s["codes"], s["scales"])
    if s["format"] == "fp8":
        return {"values": s["codes"].view(torch.float8_e4m3fn),
                "scales": s["scales"].view(torch.float8_e8m0fnu)}
    binding.mx_dequantize(s["codes"], s["scales"], s["rows"], s["dim"], "fp4", s["y"])
    return {"values": s["y"]}


def _own_rmsnorm(s):
    from q4_packed_weight_amd import binding
    binding.mx_rmsnorm(s["x"], s["residual"], s["weight"], EPS, s["rows"], s["dim"], "fp8",
                       s["residual_out"], None, s["codes"], s["scales"])
    return {"residual": s["residual_out"], "values": s["codes"].view(torch.float8_e4m3fn),
            "scales": s["scales"].view(torch.float8_e8m0fnu)}


def _own_matmul(s):
    from q4_packed_weight_amd import binding
    binding.mxfp4_matmul(s["a_codes"], s["a_scales"], s["format"], s["w_codes"], s["w_scales"],
                         s["tokens"], s["dim"], s["out"], s["y"])
    return {"y": s["y"]}


def _own_moe(s):
    from q4_packed_weight_amd import binding
    sizes = s["tokens"], s["dim"], s["ffn"], s["experts"], s["top_k"]
    if "workspace" not in s:  # kept by the program, as its other buffers are
        n = binding.mxfp4_moe_workspace_size(*sizes)
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    binding.mxfp4_moe(s["x"], s["router"], s["bias"], s["up_codes"], s["up_scales"],
                      s["down_codes"], s["down_scales"], *sizes, s["y"], s["workspace"])
    return {"y": s["y"]}


def run(state):
    if own:
        return {"quantize": _own_quantize, "rmsnorm": _own_rmsnorm, "matmul": _own_matmul,
                "moe": _own_moe}[state["op"]](state)
    return {"quantize": _plain_quantize, "rmsnorm": _plain_rmsnorm, "matmul": _plain_matmul,
            "moe": _plain_moe}[state["op"]](state)


# ---------------------------------------------------------------- 64 bits

def _exact_codes(codes, scales, fmt):
    """The held values, each from its bits."""
    if fmt == "fp4":
        n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(torch.int16)
        sign, e, m = n >> 3, (n >> 1) & 3, n & 1
        bias, frac = 1, 2.0
    else:
        n = codes.to(torch.int16)
        sign, e, m = n >> 7, (n >> 3) & 15, n & 7
        bias, frac = 7, 8.0
    m = m.double() / frac
    v = torch.where(e > 0, (1 + m) * torch.exp2(e.double() - bias), m * 2.0 ** (1 - bias))
    v = torch.where(sign > 0, -v, v)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def _exact_scaled(h, fmt):
    """(h over its block's power of two and held at the largest, the power)."""
    top, less = (6.0, 2) if fmt == "fp4" else (448.0, 8)
    amax = h.abs().unflatten(-1, (-1, 32)).amax(-1)
    e = torch.floor(torch.log2(amax.clamp(min=1e-300)))
    e = torch.where(torch.exp2(e) > amax, e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= amax, e + 1, e)
    p = torch.exp2((e - less).clamp(min=-127))
    return (h / p.repeat_interleave(32, -1)).clamp(-top, top), p


def _exact_round(v, bits, low):
    """To nearest even with `bits` bits after the leading one, none finer than 2^low."""
    step = torch.exp2((torch.floor(torch.log2(v.abs().clamp(min=1e-300))) - bits).clamp(min=low))
    return torch.round(v / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        v, p = _exact_scaled(s["x"].double(), case["format"])
        if case["format"] == "fp8":
            return {"values": _exact_round(v, 3, -9), "scales": p}
        return {"values": _exact_round(v, 1, -1) * p.repeat_interleave(32, -1)}
    if case["op"] == "rmsnorm":
        # the residual is what is stored; the values before their rounding to 8 bits
        r = (s["x"].double() + s["residual"].double())
        t = r.to(s["x"].dtype).double()
        h = t / torch.sqrt((t ** 2).sum(-1, keepdim=True) / case["dim"] + EPS)
        v, p = _exact_scaled(h * s["weight"].double(), "fp8")
        return {"residual": r, "values": v, "scales": p}
    if case["op"] == "matmul":
        a = _exact_codes(s["a_codes"], s["a_scales"], case["format"])
        w = _exact_codes(s["w_codes"], s["w_scales"], "fp4")
        return {"y": a @ w.t().contiguous()}
    x, F = s["x"].double(), case["ffn"]
    logits = x @ s["router"].double().t().contiguous() + s["bias"].double()
    rows = logits.cpu().tolist()
    shares = torch.zeros_like(logits)
    for t, row in enumerate(rows):
        best = sorted(range(len(row)), key=lambda e: (-row[e], e))[:case["top_k"]]
        z = sum(math.exp(row[e] - row[best[0]]) for e in best)
        for e in best:
            shares[t, e] = math.exp(row[e] - row[best[0]]) / z
    y = torch.zeros_like(x)
    for e in range(case["experts"]):
        who = torch.nonzero(shares[:, e]).flatten()
        if not len(who):
            continue
        gu = x[who] @ _exact_codes(s["up_codes"][e], s["up_scales"][e], "fp4").t().contiguous()
        h = gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]
        d = h @ _exact_codes(s["down_codes"][e], s["down_scales"][e], "fp4").t().contiguous()
        y[who] += shares[who, e].unsqueeze(-1) * d
    return {"y": y}
