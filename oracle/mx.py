"""CPU oracle of the microscaled (MX) operators, in float64 numpy.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  Written from the
format (OCP Microscaling Formats specification 1.0: e2m1 and e4m3 elements,
one e8m0 scale for 32 of them) and the operators' formulas; shares no code
with the GPU library.
"""
import numpy as np

BLOCK = 32


def _table(ebits, mbits, bias):
    """Non-negative values of a small float format, by code."""
    out = []
    for code in range(1 << (ebits + mbits)):
        e, m = code >> mbits, code & ((1 << mbits) - 1)
        f = m / (1 << mbits)
        out.append(f * 2.0 ** (1 - bias) if e == 0 else (1 + f) * 2.0 ** (e - bias))
    return np.array(out)


E2M1 = _table(2, 1, 1)
E4M3 = _table(4, 3, 7)
E4M3[127] = np.nan
SHIFT = {"fp4": 2, "fp8": 8}
TOP = {"fp4": 6.0, "fp8": 448.0}


def unpack(codes, fmt):
    """One code to an entry, in row order."""
    if fmt == "fp8":
        return codes
    return np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)


def pack(codes, fmt):
    if fmt == "fp8":
        return codes
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def dequantize(codes, scales, fmt):
    c = unpack(codes, fmt)
    sign = c >> (3 if fmt == "fp4" else 7)
    v = (E2M1[c & 7] if fmt == "fp4" else E4M3[c & 127]) * np.where(sign, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return v * np.repeat(s, BLOCK, axis=-1)


def _nearest(a, fmt):
    """Codes of magnitudes a, to nearest, ties to the even code."""
    t = E2M1 if fmt == "fp4" else E4M3[:127]
    a = np.minimum(a, t[-1])
    hi = np.clip(np.searchsorted(t, a, side="left"), 1, len(t) - 1)
    lo = hi - 1
    below, above = a - t[lo], t[hi] - a
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return np.where(up, hi, lo).astype(np.uint8)


def scale_bytes(amax, fmt):
    _, e = np.frexp(amax)  # amax = m 2^e, 0.5 <= m < 1
    return np.where(amax > 0, np.maximum(e - 1 - SHIFT[fmt], -127), -127) + 127


def quantize(x, fmt):
    """(codes, scales) of the rows of x."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], -1, BLOCK)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    s = scale_bytes(np.abs(b).max(-1), fmt)
    v = b / 2.0 ** (s[..., None] - 127.0)
    c = _nearest(np.abs(v), fmt) | (np.signbit(v).astype(np.uint8) << (3 if fmt == "fp4" else 7))
    c = np.where(bad[..., None], 0, c).astype(np.uint8).reshape(x.shape)
    return pack(c, fmt), np.where(bad, 255, s).astype(np.uint8)


def rmsnorm(r, weight, eps):
    r = np.asarray(r, np.float64)
    return r / np.sqrt((r * r).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def matmul(a, w):
    """(A W^T, sum of the products' magnitudes)."""
    return a @ w.T, np.abs(a) @ np.abs(w).T


def silu(g):
    return g / (1 + np.exp(-g))


def choose(logits, k):
    """Experts by descending logit, equal ones by index, NaN last."""
    key = np.where(np.isnan(logits), -np.inf, logits)
    nan = np.isnan(logits)
    return np.stack([sorted(range(len(r)), key=lambda e: (nan_r[e], -r[e], e))[:k]
                     for r, nan_r in zip(key, nan)])


def moe(x, router, bias, up, down, k, parts_error):
    """(y, error scale): the layer, and a first-order bound of what fp32-level
    rounding changes in it; tokens whose choice such rounding could change get
    an infinite bound.  up [E][2F][H], down [E][H][F]; parts_error: the
    relative error of h as the sum of bf16 parts."""
    x, router = np.asarray(x, np.float64), np.asarray(router, np.float64)
    T, H = x.shape
    F = down.shape[2]
    u = 2.0 ** -23
    logits = x @ router.T + (0 if bias is None else bias)
    # fp32 sums: 256 lanes, then a tree
    dl = (H / 256 + 24) * u * (np.abs(x) @ np.abs(router).T + np.abs(0 if bias is None else bias))
    order = choose(logits, min(k + 1, logits.shape[1]))
    y, err = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        best = order[t, :k]
        l, d = logits[t, best], dl[t, order[t]].max()
        near = order.shape[1] > k and l[-1] - logits[t, order[t, k]] <= 2 * d
        p = np.exp(l - l[0])
        p /= p.sum()
        for e, pe in zip(best, p):
            gu, s = up[e] @ x[t], np.abs(up[e]) @ np.abs(x[t])
            d_gu = (H / 128 + 24) * u * s
            g, v = gu[:F], gu[F:]
            h = silu(g) * v
            dh = np.abs(v) * 1.1 * d_gu[:F] + np.abs(silu(g)) * d_gu[F:]
            dh += (16 * u + parts_error) * np.abs(h)
            D = np.abs(down[e])
            y[t] += pe * (down[e] @ h)
            err[t] += pe * (D @ dh + ((F / 128 + 48) * u + 4 * d) * (D @ np.abs(h)))
        if near:
            err[t] = np.inf
    return y, err


def rotary(x, positions, frequencies, amplitude, rotary_dim, layout):
    """x [tokens][heads][head_dim]."""
    y = np.array(x, np.float64)
    w = np.asarray(positions, np.float64)[:, None] * np.asarray(frequencies, np.float64)
    c, s = (amplitude * np.cos(w))[:, None], (amplitude * np.sin(w))[:, None]
    h = rotary_dim // 2
    one = slice(0, h) if layout == "half" else slice(0, rotary_dim, 2)
    two = slice(h, rotary_dim) if layout == "half" else slice(1, rotary_dim, 2)
    a, b = y[..., one].copy(), y[..., two].copy()
    y[..., one], y[..., two] = a * c - b * s, b * c + a * s
    return y


def rotary_frequencies(d, base, scaling="none", factor=1.0, trained=8192.0, low=1.0, high=32.0):
    """(frequencies, amplitude), pair by pair from the definitions."""
    if scaling == "ntk" and d > 2:
        base = base * factor ** (d / (d - 2))
    f = np.array([base ** (-2 * i / d) for i in range(d // 2)])
    turns = trained * f / (2 * np.pi)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "bands":
        keep = np.clip((turns - low) / (high - low), 0, 1)
        return f * keep + f / factor * (1 - keep), 1.0
    if scaling == "yarn":
        # turns(i) = trained / (2 pi base^(2i/d)) solved for i
        at = [d / 2 * np.log(trained / (2 * np.pi * n)) / np.log(base) for n in (high, low)]
        first, last = max(np.floor(at[0]), 0), min(np.ceil(at[1]), d - 1)
        keep = 1 - np.clip((np.arange(d // 2) - first) / max(last - first, 1e-3), 0, 1)
        return f * keep + f / factor * (1 - keep), 0.1 * np.log(factor) + 1
    return f, 1.0


def attention(q, k, v, scale, sees):
    """Rows of q [rows][dim] over keys and values [keys][dim]; sees [rows][keys].
    (y, sum of the weights' shares of |v|, largest score seen, largest sum of
    |q||k| seen)."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    rows, dim = q.shape
    y, mass = np.zeros((rows, dim)), np.zeros((rows, dim))
    top, size = np.zeros(rows), np.zeros(rows)
    for r in range(rows):
        j = np.nonzero(sees[r])[0]
        if not len(j):
            continue
        x = (k[j] @ q[r]) * scale
        if np.isnan(x).any():
            y[r] = np.nan
            continue
        w = np.exp(x - x.max())
        w /= w.sum()
        y[r] = w @ v[j]
        mass[r] = w @ np.abs(v[j])
        top[r] = np.abs(x).max()
        size[r] = (np.abs(k[j]) @ np.abs(q[r])).max() * abs(scale)
    return y, mass, top, size
