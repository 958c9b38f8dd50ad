"""How many bits the MX product and the mixture-of-experts layer keep, over all
outputs together: a bound on each output is that of the worst signs, which a
form that loses half of its bits stays within.

Tolerances, from the roundings alone:
  layer_tolerance    fp32: an addition is off by at most 2^-24 of its sum, and
    the signs of the three products' roundings are even: with 3 bf16 parts of 32
    positions an instruction, 3 K / 32 additions a sum, whose squares add up over
    gate and up (2.4 of them: silu's slope reaches 1.1) and down; 8 more for the
    logits, the exponential and the weights.
    16-bit types against the rounded formula: h keeps 2^-17 of its value, so an
    output next to a border is rounded to its other side with a probability of
    2^-17 over half a step, and is a step off then; twice that.
  product_tolerance  the same, with 2^-12 for what one instruction of e4m3
    products is off (2^-11 of the largest of 128 products, which is about half
    of their sum), and for fp32 outputs the additions of two instructions a step.
"""
import numpy as np
import pytest
import torch

from gpu_util import DEV
from oracle import mx
from q4_packed_weight_amd import binding
from test_mx_paths_gpu import TYPES, U, Layer, check_matmul, gen, packed, values

gpu = pytest.mark.gpu


def layer_tolerance(kind, H, F):
    if kind == "fp32":
        return 2.0 ** -24 * (8 + np.sqrt(3 * (2.4 * H + F) / 32))
    eps = torch.finfo(TYPES[kind]).eps
    return 2 * eps * np.sqrt(2.0 ** -17 / (eps / 2))


def product_tolerance(kind, fmt, K):
    eps = torch.finfo(TYPES[kind]).eps
    if kind == "fp32":
        return 2.0 ** -24 * (1 + np.sqrt(2 * K / 128))
    return 2 * eps * np.sqrt((2.0 ** -12 if fmt == "fp8" else 2.0 ** -20) / (eps / 2))


def distance(y, ref, kind):
    """Of y from the formula's value, rounded to the type, over all outputs."""
    return float((y.double() - ref.to(TYPES[kind]).double()).norm() / ref.norm())


def formula(x, router, bias, up, down, k, x_parts=None, h_parts=None):
    """The layer in float64; x and h as sums of that many bf16 parts."""
    def cut(v, parts):
        if parts is None:
            return v
        out = torch.zeros_like(v)
        for _ in range(parts):
            out += (v - out).to(torch.bfloat16).double()
        return out
    x, F = x.double(), down.shape[2]
    top, chosen = torch.sort(x @ router.double().t().contiguous() + bias.double(), dim=-1,
                             descending=True, stable=True)
    p = torch.softmax(top[:, :k], -1)
    y = torch.zeros_like(x)
    for e in range(up.shape[0]):
        t, rank = (chosen[:, :k] == e).nonzero(as_tuple=True)
        if len(t):
            gu = cut(x[t], x_parts) @ up[e].t().contiguous()
            h = gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]
            y.index_add_(0, t, p[t, rank].unsqueeze(-1) * (cut(h, h_parts) @ down[e].t().contiguous()))
    return y


@pytest.mark.parametrize("kind,x_parts,h_parts,within", [
    ("fp32", 3, 3, True), ("fp32", 2, 3, False), ("fp32", 3, 2, False), ("fp32", 1, 1, False),
    ("bf16", 1, 2, True), ("bf16", 1, 1, False),
    ("fp16", 2, 2, True), ("fp16", 1, 2, False), ("fp16", 2, 1, False)])
@pytest.mark.parametrize("T,H,F,E,k", [(4, 256, 96, 8, 2), (6, 1056, 736, 4, 2), (3, 2048, 1024, 3, 2)])
def test_tolerances_tell_a_form_with_a_part_less(T, H, F, E, k, kind, x_parts, h_parts, within):
    g = np.random.default_rng((5, T, H))
    t = TYPES[kind]

    def weights(rows, K):
        c = g.integers(0, 256, (rows, K // 2)).astype(np.uint8)
        s = (126 - int(np.log2(K) / 2) + g.integers(0, 2, (rows, K // 32))).astype(np.uint8)
        return torch.from_numpy(mx.dequantize(c, s, "fp4"))

    x = torch.from_numpy(g.standard_normal((T, H))).to(t)
    router = torch.from_numpy(1.5 * H ** -0.5 * g.standard_normal((E, H))).to(t)
    bias = torch.from_numpy(0.3 * g.standard_normal(E)).float()
    args = x, router, bias, weights(E * 2 * F, H).view(E, 2 * F, H), weights(E * H, F).view(E, H, F), k
    y = formula(*args, x_parts, h_parts).to(t)
    d = distance(y, formula(*args), kind)
    assert bool(d <= layer_tolerance(kind, H, F)) == within, d


def check_layer(layer, **how):
    T, H, F, E, k = layer.size
    y = layer.run(**how)
    up = values(*layer.up, "fp4").view(E, 2 * F, H)
    down = values(*layer.down, "fp4").view(E, H, F)
    ref = formula(layer.x, layer.router, layer.bias, up, down, k)
    # the choice is certain where the k-th logit is clear of the next; the router's
    # sums: 256 lanes, then a tree
    r = layer.router.double().t().contiguous()
    top = torch.sort(layer.x.double() @ r + layer.bias.double(), descending=True).values
    slack = (H / 256 + 24) * U * ((layer.x.double().abs() @ r.abs()).amax(-1) + 1)
    sure = top[:, k - 1] - top[:, k] > 2 * slack if k < E else torch.ones(T, dtype=torch.bool, device=DEV)
    assert float(sure.double().mean()) > 0.5
    d = distance(y[sure], ref[sure], layer.kind)
    assert d <= layer_tolerance(layer.kind, H, F), d


# every number of columns at a time, wide and narrow tiles, long rows in pairs of
# steps, more than 16 tokens on an expert
@gpu
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T,H,F,E,k", [(1, 64, 32, 4, 1), (1, 4096, 4096, 8, 2), (3, 2048, 1024, 64, 8),
                                       (4, 256, 96, 16, 2), (13, 1056, 736, 24, 3),
                                       (24, 4128, 4160, 16, 2), (33, 1024, 2080, 16, 4),
                                       (40, 4224, 1600, 16, 2), (64, 288, 96, 1, 1),
                                       (64, 512, 256, 128, 8), (150, 96, 64, 6, 2)])
def test_layer_keeps_its_bits(T, H, F, E, k, kind):
    check_layer(Layer(T, H, F, E, k, kind))


@gpu
@pytest.mark.parametrize("T", [2, 12, 40])
def test_layer_keeps_its_bits_with_odd_scales(T):
    check_layer(Layer(T, 512, 256, 8, 2, "fp32"), odd_scales=True)


@gpu
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("M,K,N", [(1, 4096, 4096), (20, 1152, 4097), (64, 4096, 8200), (65, 1056, 300),
                                   (300, 384, 500), (1024, 512, 4096), (4096, 1056, 4096)])
def test_product_keeps_its_bits(M, K, N, fmt, kind):
    g = gen("bits", M, K, N, fmt)
    a, w = packed(g, M, K, fmt, 119, 125), packed(g, N, K, "fp4", 119, 125)
    y = torch.empty(M, N, dtype=TYPES[kind], device=DEV)
    binding.mxfp4_matmul(*a, fmt, *w, M, K, N, y)
    ref = values(*a, fmt) @ values(*w, "fp4").t().contiguous()
    d = distance(y, ref, kind)
    assert d <= product_tolerance(kind, fmt, K), d


# ------------------------------------------------------------ scale bytes of the whole range

@gpu
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("M,N", [(18, 35), (72, 35), (1026, 4112), (4104, 4112)])
def test_product_under_every_scale(M, N, fmt):
    """Rows of one scale byte each, 0 to 254, against one another.  Products
    whose sums pass fp32's range are left out; below its normals one of its
    smallest normals is allowed."""
    K = 256
    g = gen("scales", M, N, fmt)
    (ac, as_), (wc, ws) = packed(g, M, K, fmt), packed(g, N, K, "fp4")
    for s in (as_, ws):
        n = s.shape[0]
        s.copy_((torch.arange(n, device=DEV) * 254 // (min(n, 255) - 1) % 255).to(torch.uint8).unsqueeze(-1))
        s[0], s[1], s[2], s[n - 1] = 0, 1, 254, 253
    a, w = values(ac, as_, fmt), values(wc, ws, "fp4")
    y = torch.empty(M, N, device=DEV)
    binding.mxfp4_matmul(ac, as_, fmt, wc, ws, M, K, N, y)
    ref, size = a @ w.t().contiguous(), a.abs() @ w.abs().t().contiguous()
    bound = 2.0 ** -24 * ref.abs() + (K / 128 + 24) * U * size + 2.0 ** -126
    fits = size < 2.0 ** 127
    assert bool(((y.double() - ref).abs() <= bound)[fits].all())


@gpu
@pytest.mark.parametrize("H,F", [(256, 128), (288, 160)])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("T", [1, 6, 40])
@pytest.mark.parametrize("which", ["up", "down"])
def test_layer_under_the_smallest_scales(which, T, kind, H, F):
    """Weights of scale bytes 0 and 1 (2^-127 and 2^-126) against activations
    that bring their products back to ordinary size."""
    layer = Layer(T, H, F, 8, 2, kind)
    if which == "up":
        layer.x = (layer.x.double() * 2.0 ** 120).to(TYPES[kind])
        layer.router = (layer.router.double() * 2.0 ** -120).to(TYPES[kind])
        layer.up[1].copy_(layer.up[1] % 2)
    else:
        layer.up[1].add_(58)
        layer.down[1].copy_(layer.down[1] % 2)
    check_layer(layer)


# ------------------------------------------------------------ the longest rows

@gpu
@pytest.mark.parametrize("K", [(1 << 22) + 32, (1 << 22) + 128])
@pytest.mark.parametrize("M,fmt", [(65, "fp8"), (130, "fp4")])
def test_product_of_more_tokens_and_positions_than_tiles_take(M, K, fmt):
    check_matmul(M, K, 33, fmt, "fp32")


@gpu
@pytest.mark.parametrize("H,F", [(1 << 20, 32), (32, 1 << 20)])
def test_layer_whose_slots_fill_31_bits(H, F):
    """60 tokens run as 56 and 4, so that the offsets of a group stay in range."""
    Layer(60, H, F, 6, 6, "fp32").check()
