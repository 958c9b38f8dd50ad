"""Attention over a quantised cache: what is measured, and the plain forms.

The keys and values of a layer lie in pages of a pool, in blocks of 32 values of
a head with one power of two (MXFP4 or MXFP8, as perf/operators.py has them):
codes [pages][heads][page size][bytes of a head], scales [..][head_dim / 32];
slot = page * page size + place.

  rotary     the pairs (a, b) of the first rotary_dim values of a head turn by
             position * frequency: (a cos - b sin, b cos + a sin) * amplitude;
             half layout: i and i + rotary_dim / 2, interleaved: 2i and 2i + 1
  cache      rows of keys and values to the blocks of their slots, and back
  attention  the queries of each sequence over its first `keys` cached tokens:
             softmax(scale q k) v, several query heads to a key head; causal:
             the last query sees the last key, one before it one less, and no
             more than `window` keys where that is not 0
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
FP4_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decoding step late in a long context
        {"name": "rotary 1x40x128", "op": "rotary", "type": "bf16", "tokens": 1, "heads": 40,
         "head_dim": 128, "rotary_dim": 128, "layout": "half", "scaling": "none", "far": 131072},
        # a prompt's queries and keys, frequencies stretched for long contexts
        {"name": "rotary 4096x40x128", "op": "rotary", "type": "bf16", "tokens": 4096, "heads": 40,
         "head_dim": 128, "rotary_dim": 128, "layout": "half", "scaling": "yarn", "far": 65536},
        # pairs of neighbours in two thirds of a head, a ragged batch
        {"name": "rotary part 333x15x96", "op": "rotary", "type": "fp16", "tokens": 333,
         "heads": 15, "head_dim": 96, "rotary_dim": 64, "layout": "interleaved",
         "scaling": "bands", "far": 32768},
        # the new tokens of a decoding batch
        {"name": "cache write fp8 64x8x128", "op": "cache", "do": "write", "type": "bf16",
         "format": "fp8", "tokens": 64, "heads": 8, "head_dim": 128, "page": 16, "pages": 512},
        # a chunk of a prompt written and read back, odd sizes
        {"name": "cache fp4 2049x5x96", "op": "cache", "do": "both", "type": "fp16",
         "format": "fp4", "tokens": 2049, "heads": 5, "head_dim": 96, "page": 64, "pages": 40},
        # a cached prefix read back as a whole
        {"name": "cache read fp8 32768x8x128", "op": "cache", "do": "read", "type": "bf16",
         "format": "fp8", "tokens": 32768, "heads": 8, "head_dim": 128, "page": 64, "pages": 600},
        # one sequence, one token: latency
        {"name": "attention 1 token, 1000 keys", "op": "attention", "type": "bf16",
         "format": "fp8", "seqs": 1, "queries": 1, "keys": 1000, "kv_heads": 8, "group": 4,
         "head_dim": 128, "page": 16, "causal": True, "window": 0, "mixed": False},
        # a decoding batch of sequences of all lengths
        {"name": "attention 64 tokens, to 8192 keys", "op": "attention", "type": "bf16",
         "format": "fp8", "seqs": 64, "queries": 1, "keys": 8192, "kv_heads": 8, "group": 4,
         "head_dim": 128, "page": 16, "causal": True, "window": 0, "mixed": True},
        # two long contexts in 4 bits
        {"name": "attention 2 tokens, to 131072 keys fp4", "op": "attention", "type": "bf16",
         "format": "fp4", "seqs": 2, "queries": 1, "keys": 131072, "kv_heads": 8, "group": 8,
         "head_dim": 128, "page": 64, "causal": True, "window": 0, "mixed": True},
        # a chunk of a long prompt
        {"name": "attention 2048 of 8192", "op": "attention", "type": "bf16", "format": "fp8",
         "seqs": 1, "queries": 2048, "keys": 8192, "kv_heads": 8, "group": 4, "head_dim": 128,
         "page": 64, "causal": True, "window": 0, "mixed": False},
        # chunks and single tokens in one batch, a sliding window, odd sizes
        {"name": "attention mixed batch, window", "op": "attention", "type": "fp16",
         "format": "fp4", "seqs": 13, "queries": 301, "keys": 5000, "kv_heads": 5, "group": 3,
         "head_dim": 96, "page": 32, "causal": True, "window": 1000, "mixed": True},
        # cross attention: each sequence's tokens over all of an encoder's states
        {"name": "attention cross 4x187 over 1500", "op": "attention", "type": "fp32",
         "format": "fp8", "seqs": 4, "queries": 187, "keys": 1500, "kv_heads": 16, "group": 1,
         "head_dim": 64, "page": 128, "causal": False, "window": 0, "mixed": False},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["rotary", "cache", "attention", "attention"])
    case = {"op": op, "type": rng.choice(["fp32", "bf16", "fp16"]), "head_dim": 32 * rng.randint(1, 8)}
    D = case["head_dim"]
    if op == "rotary":
        case["heads"] = _log(rng, 1, 64)
        case["tokens"] = min(_log(rng, 1, 8192), (1 << 24) // (case["heads"] * D))
        case["rotary_dim"] = D if rng.random() < 0.5 else 2 * rng.randint(1, D // 2)
        case["layout"] = rng.choice(["half", "interleaved"])
        case["scaling"] = rng.choice(["none", "linear", "ntk", "yarn", "bands"])
        case["far"] = _log(rng, 8192, 1 << 20)
        return case
    case["format"] = rng.choice(["fp4", "fp8"])
    case["page"] = rng.choice([16, 32, 64, 128, 256])
    if op == "cache":
        case["heads"] = _log(rng, 1, 32)
        case["do"] = rng.choice(["both", "read"] if case["format"] == "fp4" else ["write", "both", "read"])
        case["tokens"] = min(_log(rng, 1, 32768), (1 << 24) // (case["heads"] * D))
        case["pages"] = case["tokens"] // case["page"] + rng.randint(1, 40)
        return case
    case["kv_heads"], case["group"] = rng.randint(1, 8), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    case["seqs"], case["mixed"] = _log(rng, 1, 64), rng.random() < 0.5
    room = (1 << 27) // (case["seqs"] * case["kv_heads"] * D)  # of the cache
    case["keys"] = min(_log(rng, 1, 65536), room)
    case["causal"] = rng.random() < 0.75
    case["window"] = _log(rng, 1, 8192) if case["causal"] and rng.random() < 0.25 else 0
    rows = case["seqs"] * case["kv_heads"] * case["group"]
    most = (1 << 34) // (rows * case["keys"] * D)
    case["queries"] = 1 if rng.random() < 0.5 else max(1, min(_log(rng, 1, 1024), most))
    if case["causal"]:
        case["queries"] = min(case["queries"], case["keys"])
    return case


def _counts(case):
    """(queries, keys) of each sequence; a batch is the same at every seed."""
    if not case["mixed"]:
        return [(case["queries"], case["keys"])] * case["seqs"]
    r = random.Random(case["seqs"] * 1000003 + case["keys"])
    out = []
    for _ in range(case["seqs"]):
        nk = r.randint((case["keys"] + 7) // 8, case["keys"])
        # about a third of a batch of chunks is at its single tokens
        nq = 1 if r.random() < 0.35 else r.randint(1, case["queries"])
        out.append((min(nq, nk), nk))
    return out


def work(case):
    size, D = {"fp32": 4, "bf16": 2, "fp16": 2}[case["type"]], case["head_dim"]
    code = {"fp4": 0.5, "fp8": 1.0}[case.get("format", "fp8")] + 1 / 32
    if case["op"] == "rotary":
        n = case["tokens"] * case["heads"] * D
        return {"bytes": 2 * n * size + 8 * (case["tokens"] + case["rotary_dim"] // 2),
                "flops": case["tokens"] * case["heads"] * 3 * case["rotary_dim"]}
    if case["op"] == "cache":
        n = 2 * case["tokens"] * case["heads"] * D
        passes = 2 if case["do"] == "both" else 1
        # written and read back: the codes are an output, no second reading of them is needed
        return {"bytes": n * (passes * size + code) + 8 * case["tokens"], "flops": 2 * passes * n}
    cached = pairs = tokens = 0
    for nq, nk in _counts(case):
        tokens += nq
        w = case["window"] or nk
        if case["causal"]:
            cached += min(nk, w + nq - 1)
            pairs += sum(min(nk - nq + i + 1, w) for i in range(nq))
        else:
            cached += nk
            pairs += nq * nk
    heads = case["kv_heads"] * case["group"]
    return {"bytes": 2 * cached * case["kv_heads"] * D * code + 2 * tokens * heads * D * size,
            "flops": 4 * pairs * heads * D}


# ---------------------------------------------------------------- inputs

def _frequencies(case):
    """(radians a position of each pair, amplitude), base 10000, for contexts four
    times as long as the 8192 trained on."""
    d, base, factor, trained = case["rotary_dim"], 10000.0, 4.0, 8192
    if case["scaling"] == "ntk" and d > 2:
        base *= factor ** (d / (d - 2))
    f = [base ** (-2 * i / d) for i in range(d // 2)]
    if case["scaling"] == "linear":
        return [x / factor for x in f], 1.0
    if case["scaling"] == "bands":  # by turns over the trained context, 1 to 4
        keep = [min(1.0, max(0.0, (trained * x / (2 * math.pi) - 1) / 3)) for x in f]
        return [x * (k + (1 - k) / factor) for x, k in zip(f, keep)], 1.0
    if case["scaling"] == "yarn":  # by index, between those of 32 turns and of 1

        def at(turns):
            return d * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(at(32)), 0), min(math.ceil(at(1)), d - 1)
        keep = [1 - min(1.0, max(0.0, (i - low) / max(high - low, 1e-3))) for i in range(d // 2)]
        return [x * (k + (1 - k) / factor) for x, k in zip(f, keep)], 0.1 * math.log(factor) + 1
    return f, 1.0


def _rng(seed):
    g = torch.Generator(DEV)
    g.manual_seed(int(seed))
    return g


def _rows(g, tokens, heads, D):
    """Normal values with a spread of channel sizes, a few of them large."""
    channel = torch.exp(0.5 * torch.randn(heads, D, generator=g, device=DEV))
    return torch.randn(tokens, heads, D, generator=g, device=DEV) * channel


def _pool(g, case, heads, filled):
    """Codes and scales of the pages of keys, then those of values."""
    D, fmt, pages, page = case["head_dim"], case["format"], case["pages"], case["page"]
    out = []
    for _ in range(2):
        codes = torch.zeros(pages, heads, page, D if fmt == "fp8" else D // 2, dtype=torch.uint8,
                            device=DEV)
        scales = torch.zeros(pages, heads, page, D // 32, dtype=torch.uint8, device=DEV)
        step = max(1, (1 << 25) // (heads * page * D))
        for a in range(0, pages if filled else 0, step):
            n = min(step, pages - a)
            x = _rows(g, n * page, heads, D).view(n, page, heads, D).transpose(1, 2)
            c, t = _quantize(x, fmt)
            codes[a:a + n] = _pack(c) if fmt == "fp4" else c.view(torch.uint8)
            scales[a:a + n] = t
        out += [codes, scales]
    return out


def prepare(case, seed):
    dtype, D = TYPES[case["type"]], case["head_dim"]
    s, g = dict(case), _rng(seed)
    if case["op"] == "rotary":
        T, H = case["tokens"], case["heads"]
        # rows of a projection, whose values (as many as a quarter of these heads) stay
        s["rows"] = _rows(g, T, H + (H + 3) // 4, D).flatten(1).to(dtype)
        first = torch.randint(0, case["far"] - T, (1,), generator=g, device=DEV)
        s["positions"] = first + torch.arange(T, device=DEV)
        f, s["amplitude"] = _frequencies(case)
        s["frequencies"] = torch.tensor(f, dtype=torch.float64, device=DEV)
        s["y"] = torch.empty(T, H * D, dtype=dtype, device=DEV)
        return s
    if case["op"] == "cache":
        T, H = case["tokens"], case["heads"]
        s["pool"] = _pool(g, case, H, case["do"] == "read")
        n = case["pages"] * case["page"]
        if case["do"] == "write":  # a token each of as many sequences
            s["slots"] = torch.randperm(n, generator=g, device=DEV)[:T]
        else:  # a sequence's pages, in no order
            order = torch.randperm(case["pages"], generator=g, device=DEV)
            t = torch.arange(T, device=DEV)
            s["slots"] = order[t // case["page"]] * case["page"] + t % case["page"]
        s["k"], s["v"] = (_rows(g, T, H, D).flatten(1).to(dtype) for _ in range(2))
        s["k_back"], s["v_back"] = (torch.empty(T, H * D, dtype=dtype, device=DEV)
                                    for _ in range(2))
        return s
    counts = _counts(case)
    need = [-(-nk // case["page"]) for _, nk in counts]
    s["pages"] = sum(need) + 3
    s["pool"] = _pool(g, s, case["kv_heads"], True)
    order = torch.randperm(s["pages"], generator=g, device=DEV).int()
    s["table"] = torch.zeros(len(counts), max(need), dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(need):
        s["table"][i, :n] = order[at:at + n]
        at += n
    s["counts"] = counts
    starts = [0]
    for nq, _ in counts:
        starts.append(starts[-1] + nq)
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    s["lengths"] = torch.tensor([nk for _, nk in counts], dtype=torch.int32, device=DEV)
    s["max_queries"] = max(nq for nq, _ in counts)
    H = case["kv_heads"] * case["group"]
    s["q"] = (_rows(g, starts[-1], H, D) * 0.8).flatten(1).to(dtype)
    s["y"] = torch.empty_like(s["q"])
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
    return (code + 8 * torch.signbit(v)).to(torch.uint8), scales


def _pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _values(codes, scales, fmt):
    """What codes and scales stand for, in 32 bits."""
    if fmt == "fp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        one = torch.tensor(FP4_VALUES + tuple(-x for x in FP4_VALUES), device=codes.device)
        pair = torch.stack([one.repeat(16), one.repeat_interleave(16)], -1)
        v = pair[codes.int()].flatten(-2)
    power = torch.ldexp(torch.ones((), device=scales.device), scales.int() - 127)
    return (v.unflatten(-1, (-1, 32)) * power.unsqueeze(-1)).flatten(-2)


def _plain_rotary(s):
    T, H, D, R = s["tokens"], s["heads"], s["head_dim"], s["rotary_dim"]
    x = s["rows"][:, :H * D].float().view(T, H, D)
    angle = s["positions"].double().unsqueeze(-1) * s["frequencies"]
    cos = (torch.cos(angle) * s["amplitude"]).float().unsqueeze(1)
    sin = (torch.sin(angle) * s["amplitude"]).float().unsqueeze(1)
    if s["layout"] == "half":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return {"y": torch.cat([turned, x[..., R:]], -1).flatten(1).to(s["y"].dtype)}


def _plain_cache(s):
    T, H, D, fmt = s["tokens"], s["heads"], s["head_dim"], s["format"]
    at, place = s["slots"] // s["page"], s["slots"] % s["page"]
    out = {}
    for i, name in ((0, "k"), (2, "v")):
        codes, scales = s["pool"][i], s["pool"][i + 1]
        if s["do"] != "read":
            c, t = _quantize(s[name].view(T, H, D), fmt)
            codes[at, :, place] = _pack(c) if fmt == "fp4" else c.view(torch.uint8)
            scales[at, :, place] = t
        if s["do"] != "write":
            out[name] = _values(codes[at, :, place], scales[at, :, place], fmt).flatten(1).to(
                s[name].dtype)
        else:
            out[name] = codes.view(torch.float8_e4m3fn)
            out[name + " scales"] = scales.view(torch.float8_e8m0fnu)
    return out


def _plain_attention(s):
    Hk, G, D = s["kv_heads"], s["group"], s["head_dim"]
    at, out = 0, []
    for i, (nq, nk) in enumerate(s["counts"]):
        pages = s["table"][i, :-(-nk // s["page"])].long()
        k, v = (_values(s["pool"][j][pages], s["pool"][j + 1][pages], s["format"])
                .transpose(0, 1).flatten(1, 2)[:, :nk] for j in (0, 2))
        q = s["q"][at:at + nq].float().view(nq, Hk, G, D).permute(1, 0, 2, 3).flatten(1, 2)
        scores = torch.matmul(q, k.transpose(1, 2).contiguous()) * D ** -0.5
        if s["causal"]:
            last = torch.arange(nk - nq, nk, device=DEV).repeat_interleave(G).unsqueeze(-1)
            key = torch.arange(nk, device=DEV)
            hidden = key > last
            if s["window"]:
                hidden = hidden | (key <= last - s["window"])
            scores.masked_fill_(hidden, -math.inf)
        scores -= scores.amax(-1, keepdim=True)
        scores.exp_()
        y = torch.matmul(scores, v) / scores.sum(-1, keepdim=True)
        out.append(y.view(Hk, nq, G, D).permute(1, 0, 2, 3).reshape(nq, -1))
        at += nq
    return {"y": torch.cat(out).to(s["y"].dtype)}


# ---------------------------------------------------------------- the framework's calls

def _own_rotary(s):
    from q4_packed_weight_amd import binding
    H, D = s["heads"], s["head_dim"]
    binding.mx_rotary(s["rows"][:, :H * D], s["positions"], s["frequencies"], s["amplitude"],
                      s["tokens"], H, D, s["rotary_dim"], s["layout"], s["y"])
    return {"y": s["y"]}


def _own_cache(s):
    from q4_packed_weight_amd import binding
    sizes = s["tokens"], s["heads"], s["head_dim"], s["format"]
    if s["do"] != "read":
        binding.mx_cache_write(s["k"], s["v"], s["slots"], *sizes, *s["pool"], s["pages"],
                               s["page"])
    if s["do"] == "write":
        k, k_scales, v, v_scales = s["pool"]
        return {"k": k.view(torch.float8_e4m3fn), "k scales": k_scales.view(torch.float8_e8m0fnu),
                "v": v.view(torch.float8_e4m3fn), "v scales": v_scales.view(torch.float8_e8m0fnu)}
    binding.mx_cache_read(s["slots"], *sizes, *s["pool"], s["pages"], s["page"], s["k_back"],
                          s["v_back"])
    return {"k": s["k_back"], "v": s["v_back"]}


def _own_attention(s):
    from q4_packed_weight_amd import binding
    heads = s["kv_heads"] * s["group"], s["kv_heads"], s["head_dim"]
    tokens, (seqs, width) = s["q"].shape[0], s["table"].shape
    if "workspace" not in s:  # kept by the program, as its other buffers are
        n = binding.mx_attention_workspace_size(tokens, *heads, seqs, width, s["page"],
                                                s["max_queries"])
        s["workspace"] = torch.zeros(n, dtype=torch.uint8, device=DEV)
    binding.mx_attention(s["q"], s["starts"], s["lengths"], s["table"], tokens, *heads, seqs,
                         width, s["max_queries"], s["head_dim"] ** -0.5, s["causal"], s["window"],
                         s["format"], *s["pool"], s["pages"], s["page"], s["y"], s["workspace"])
    return {"y": s["y"]}


def run(state):
    if own:
        return {"rotary": _own_rotary, "cache": _own_cache,
                "attention": _own_attention}[state["op"]](state)
    return {"rotary": _plain_rotary, "cache": _plain_cache,
            "attention": _plain_attention}[state["op"]](state)


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


def _exact_blocks(h, fmt):
    """(what is held in place of h before its block's power, the power)."""
    top, less, bits, low = (6.0, 2, 1, -1) if fmt == "fp4" else (448.0, 8, 3, -9)
    amax = h.abs().unflatten(-1, (-1, 32)).amax(-1)
    e = torch.floor(torch.log2(amax.clamp(min=1e-300)))
    e = torch.where(torch.exp2(e) > amax, e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= amax, e + 1, e)
    p = torch.exp2((e - less).clamp(min=-127))
    v = (h / p.repeat_interleave(32, -1)).clamp(-top, top)
    step = torch.exp2((torch.floor(torch.log2(v.abs().clamp(min=1e-300))) - bits).clamp(min=low))
    return torch.round(v / step) * step, p


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        T, H, D, R = case["tokens"], case["heads"], case["head_dim"], case["rotary_dim"]
        x = s["rows"].double()[:, :H * D].reshape(T, H, D)
        turn = torch.polar(torch.full((T, R // 2), float(s["amplitude"]), dtype=torch.float64,
                                      device=DEV),
                           torch.outer(s["positions"].double(), s["frequencies"]))
        y = x.clone()
        halves = case["layout"] == "half"
        one = slice(0, R // 2) if halves else slice(0, R, 2)
        two = slice(R // 2, R) if halves else slice(1, R, 2)
        z = torch.complex(x[..., one].contiguous(), x[..., two].contiguous()) * turn.unsqueeze(1)
        y[..., one], y[..., two] = z.real, z.imag
        return {"y": y.flatten(1)}
    if case["op"] == "cache":
        T, H, D, page = case["tokens"], case["heads"], case["head_dim"], case["page"]
        out = {}
        for i, name in ((0, "k"), (2, "v")):
            if case["do"] == "read":
                codes = s["pool"][i].transpose(1, 2).flatten(0, 1)[s["slots"]]
                scales = s["pool"][i + 1].transpose(1, 2).flatten(0, 1)[s["slots"]]
                out[name] = _exact_codes(codes, scales, case["format"]).flatten(1)
                continue
            v, p = _exact_blocks(s[name].double().view(T, H, D), case["format"])
            if case["do"] == "both":
                out[name] = (v * p.repeat_interleave(32, -1)).flatten(1)
                continue
            pool = torch.zeros(case["pages"] * page, H, D, dtype=torch.float64, device=DEV)
            scales = torch.full((case["pages"] * page, H, D // 32), 2.0 ** -127,
                                dtype=torch.float64, device=DEV)
            pool[s["slots"]], scales[s["slots"]] = v, p
            out[name] = pool.view(-1, page, H, D).transpose(1, 2).contiguous()
            out[name + " scales"] = scales.view(-1, page, H, D // 32).transpose(1, 2).contiguous()
        return out
    Hk, G, D, page = case["kv_heads"], case["group"], case["head_dim"], case["page"]
    y = torch.zeros(s["q"].shape[0], Hk, G, D, dtype=torch.float64, device=DEV)
    starts = s["starts"].tolist()
    for i, (nq, nk) in enumerate(s["counts"]):
        rows = s["q"][starts[i]:starts[i + 1]].double().view(nq, Hk, G, D)
        table = s["table"][i].long()
        for h in range(Hk):
            k, v = (_exact_codes(s["pool"][j][table, h].flatten(0, 1)[:nk],
                                 s["pool"][j + 1][table, h].flatten(0, 1)[:nk], case["format"])
                    for j in (0, 2))
            for a in range(0, nq, 512):  # some queries at a time
                n = min(512, nq - a)
                z = rows[a:a + n, h].reshape(n * G, D) @ k.t().contiguous() / math.sqrt(D)
                if case["causal"]:
                    seen = nk - nq + a + torch.arange(n, device=DEV).repeat_interleave(G) + 1
                    back = seen.unsqueeze(-1) - torch.arange(nk, device=DEV)  # 1: the query's own
                    z[(back < 1) | (back > (case["window"] or nk))] = -math.inf
                p = torch.exp(z - torch.logsumexp(z, -1, keepdim=True))
                y[starts[i] + a:starts[i] + a + n, h] = (p @ v).view(n, G, D)
    return {"y": y.view(-1, Hk * G * D)}
