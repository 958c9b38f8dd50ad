"""The MX product and mixture-of-experts kernels where their forms change over:
tile sizes, few and many tokens, aligned and unaligned scales, whole and partial
tiles, columns at a time, long rows.  The reference is the formula in float64,
computed on the GPU from the values the codes stand for.

Bounds as in test_mx_gpu.py: half a step of the output's type, 2^-23 for each
addition of a sum of the kernel's shape times the magnitudes added, and for one
instruction of e4m3 products 2^-10 of the largest of 128 (twice 2^-11, the
steps may be cut elsewhere), which is at most 2^-10 times the sum of them.
"""
import zlib

import numpy as np
import pytest
import torch

from oracle import mx
from q4_packed_weight_amd import binding
from gpu_util import DEV

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
U = 2.0 ** -23
GUARD = 64


def gen(*seed):
    g = torch.Generator(DEV)
    g.manual_seed(zlib.crc32(repr(seed).encode()))
    return g


def packed(g, rows, K, fmt, low=123, high=129):
    """Random codes (no e4m3 NaN) and scales on the GPU."""
    c = torch.randint(0, 256, (rows, K // 2 if fmt == "fp4" else K), generator=g, device=DEV,
                      dtype=torch.uint8)
    if fmt == "fp8":
        c = torch.where((c & 127) == 127, c - 1, c)
    s = torch.randint(low, high, (rows, K // 32), generator=g, device=DEV, dtype=torch.uint8)
    return c, s


E2M1 = torch.tensor(np.concatenate([mx.E2M1, -mx.E2M1]))
E4M3 = torch.tensor(np.concatenate([mx.E4M3, -mx.E4M3]))


def values(c, s, fmt):
    """float64 values of codes and scales, on the GPU."""
    if fmt == "fp4":
        v = E2M1.to(DEV)[torch.stack([c & 15, c >> 4], -1).flatten(-2).int()]
    else:
        v = E4M3.to(DEV)[c.int()]
    p = torch.exp2(s.double() - 127)
    p = torch.where(s == 255, torch.full_like(p, float("nan")), p)
    return v * p.repeat_interleave(32, -1)


def guarded(shape, t, shift=0):
    """(whole buffer, view of `shape`, `shift` elements past a 16-byte address)."""
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * GUARD + shift,), float("nan"), dtype=t, device=DEV)
    return buf, buf[GUARD + shift:GUARD + shift + n].view(shape)


def untouched(buf, shape, shift=0):
    n = int(np.prod(shape))
    return bool(buf[:GUARD + shift].isnan().all() and buf[GUARD + shift + n:].isnan().all())


def odd(t):
    """The same bytes from an odd address on."""
    b = torch.empty(t.numel() + 1, dtype=torch.uint8, device=DEV)
    b[1:] = t.flatten()
    return b[1:]


def check_matmul(M, K, N, fmt, kind, shift=0, odd_scales=False):
    g = gen(M, K, N, fmt)
    (ac, as_), (wc, ws) = packed(g, M, K, fmt), packed(g, N, K, "fp4")
    a, w = values(ac, as_, fmt), values(wc, ws, "fp4")
    buf, y = guarded((M, N), TYPES[kind], shift)
    if odd_scales:
        as_, ws = odd(as_), odd(ws)
    binding.mxfp4_matmul(ac, as_, fmt, wc, ws, M, K, N, y)
    ref = a @ w.t().contiguous()
    size = a.abs() @ w.abs().t().contiguous()
    bound = torch.finfo(TYPES[kind]).eps / 2 * ref.abs() + (K / 128 + 24) * U * size
    if kind != "fp32" and fmt == "fp8":
        bound += 2.0 ** -10 * size
    if kind == "fp16":
        bound += 2.0 ** -25
    ok = (y.double() - ref).abs() <= bound
    # what rounds past the type's largest value is an infinity
    top = torch.finfo(TYPES[kind]).max * (1 + torch.finfo(TYPES[kind]).eps / 4)
    ok |= y.isinf() & (y.double() * ref > 0) & (ref.abs() + bound >= top)
    assert bool(ok.all())
    assert untouched(buf, (M, N), shift)


# few tokens: 16, 32 and 64 columns, one and two tiles of rows, both kinds of
# scales; the steps of a row shared out among waves unevenly
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("M", [1, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("K,N", [(128, 4096), (1152, 4097), (416, 4100), (4608, 70), (640, 8193)])
def test_few_tokens(M, K, N, fmt):
    check_matmul(M, K, N, fmt, "fp32")


@pytest.mark.parametrize("M", [1, 20, 40, 70])
@pytest.mark.parametrize("K", [65536, 33056])
def test_long_rows(M, K):
    check_matmul(M, K, 45, "fp8", "fp32")


# 64x64, 128x128 and 256x256 tiles, whole and partial
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("M,K,N", [(65, 256, 512), (128, 544, 1000), (1024, 384, 4096),
                                   (1030, 96, 4104), (4096, 128, 4096), (4095, 160, 4100),
                                   (3000, 1056, 5001)])
def test_many_tokens(M, K, N, fmt, kind):
    check_matmul(M, K, N, fmt, kind)


@pytest.mark.parametrize("M,K,N", [(48, 256, 8200), (200, 256, 500), (1024, 256, 4096),
                                   (4096, 256, 4096)])
@pytest.mark.parametrize("shift,odd_scales", [(1, False), (0, True), (4, True)])
def test_many_tokens_unaligned(M, K, N, shift, odd_scales):
    check_matmul(M, K, N, "fp8", "bf16", shift, odd_scales)


@pytest.mark.parametrize("M,N", [(1024, 4096), (4096, 4100)])
def test_many_tokens_nan_blocks_stay_in_their_row(M, N):
    K = 160
    g = gen(M, N)
    (ac, as_), (wc, ws) = packed(g, M, K, "fp8"), packed(g, N, K, "fp4")
    as_[M // 2, 4] = 255
    ws[N - 1, 0] = 255
    y = torch.empty(M, N, device=DEV)
    binding.mxfp4_matmul(ac, as_, "fp8", wc, ws, M, K, N, y)
    want = torch.zeros(M, N, dtype=torch.bool, device=DEV)
    want[M // 2] = want[:, N - 1] = True
    assert torch.equal(y.isnan(), want)


# ------------------------------------------------------------ moe

class Layer:
    def __init__(self, T, H, F, E, k, kind, seed=0):
        self.g, t = gen(T, H, F, E, k, seed), TYPES[kind]
        self.size, self.kind = (T, H, F, E, k), kind
        self.x = torch.randn(T, H, generator=self.g, device=DEV).to(t)
        self.router = (1.5 * H ** -0.5 * torch.randn(E, H, generator=self.g, device=DEV)).to(t)
        self.bias = 0.3 * torch.randn(E, generator=self.g, device=DEV)
        up, down = 126 - int(np.log2(H) / 2), 126 - int(np.log2(F) / 2)
        self.up = packed(self.g, E * 2 * F, H, "fp4", up, up + 2)
        self.down = packed(self.g, E * H, F, "fp4", down, down + 2)
        self.workspace = torch.full((binding.mxfp4_moe_workspace_size(*self.size),), 0xFF,
                                    dtype=torch.uint8, device=DEV)

    def run(self, y=None, odd_scales=False):
        T, H = self.size[:2]
        y = torch.empty(T, H, dtype=TYPES[self.kind], device=DEV) if y is None else y
        us, ds = self.up[1], self.down[1]
        if odd_scales:
            us, ds = odd(us), odd(ds)
        binding.mxfp4_moe(self.x, self.router, self.bias, self.up[0], us, self.down[0], ds,
                          *self.size, y, self.workspace)
        return y

    def reference(self):
        """The formula, and a bound on what the kernels may differ by: `unit`
        for each of a sum's roundings in the way from x to y (the parts that x
        and h enter as keep 24 bits for fp32, 16 otherwise), times the
        magnitudes that the products add."""
        T, H, F, E, k = self.size
        unit = 2.0 ** -24 if self.kind == "fp32" else 2.0 ** -17
        x = self.x.double()
        logits = x @ self.router.double().t().contiguous() + self.bias.double()
        top, chosen = torch.sort(logits, dim=-1, descending=True, stable=True)
        p = torch.softmax(top[:, :k], -1)
        # fp32 logits: a choice is only certain where the k-th is clear of the next
        slack = (H / 8 + 24) * U * (x.abs() @ self.router.double().abs().t().contiguous()).amax(-1)
        clear = (top[:, k - 1] - top[:, k] > 2 * slack) if k < E else torch.ones_like(slack, dtype=torch.bool)
        y, err = torch.zeros_like(x), torch.zeros_like(x)
        up_c, up_s = self.up[0].view(E, 2 * F, -1), self.up[1].view(E, 2 * F, -1)
        dn_c, dn_s = self.down[0].view(E, H, -1), self.down[1].view(E, H, -1)
        # roundings of a product's sum: its steps, the waves, the parts
        n_up, n_down = H / 32 + 16, F / 32 + 16
        for e in range(E):
            at = (chosen[:, :k] == e).nonzero()
            if not len(at):
                continue
            t, share = at[:, 0], p[at[:, 0], at[:, 1]].unsqueeze(-1)
            u, d = values(up_c[e], up_s[e], "fp4"), values(dn_c[e], dn_s[e], "fp4")
            gu = x[t] @ u.t().contiguous()
            off = (unit + n_up * U) * (x[t].abs() @ u.abs().t().contiguous())
            gate, lin = gu[:, :F], gu[:, F:]
            act = gate * torch.sigmoid(gate)
            h = act * lin
            # |silu'| <= 1.1; 8 roundings of exp, quotient and products
            dh = (1.1 * off[:, :F] * lin.abs() + act.abs() * off[:, F:] + 1.1 * off[:, :F] * off[:, F:]
                  + (8 * U + unit) * h.abs())
            o = h @ d.t().contiguous()
            do = dh @ d.abs().t().contiguous() + n_down * U * (h.abs() @ d.abs().t().contiguous())
            # the weights: two softmax weights' worth of the logits' slack
            y.index_add_(0, t, share * o)
            err.index_add_(0, t, share * do + share * o.abs() * (2 * slack[t].unsqueeze(-1) + 24 * U))
        return y, err, clear

    def check(self, **how):
        T, H = self.size[:2]
        buf, y = guarded((T, H), TYPES[self.kind])
        self.run(y, **how)
        ref, err, clear = self.reference()
        bound = torch.finfo(TYPES[self.kind]).eps / 2 * ref.abs() + err
        if self.kind == "fp16":
            bound += 2.0 ** -25
        assert float(clear.double().mean()) > 0.5  # most tokens are looked at
        assert bool((((y.double() - ref).abs() <= bound) | ~clear.unsqueeze(-1)).all())
        assert untouched(buf, (T, H))


# tokens around 4 (four columns at a time) and around two an expert (eight)
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T,H,F,E,k", [(4, 256, 96, 16, 2), (5, 256, 96, 16, 2), (16, 256, 96, 16, 2),
                                       (17, 256, 96, 16, 2), (5, 1056, 160, 3, 3),
                                       (64, 128, 32, 128, 16), (64, 288, 96, 1, 1)])
def test_moe_columns(T, H, F, E, k, kind):
    Layer(T, H, F, E, k, kind).check()


# wide, middle and narrow tiles; long rows, whose weights come in pairs of steps
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T,H,F,E,k", [(32, 4096, 96, 256, 16), (9, 512, 4096, 32, 8),
                                       (24, 4128, 4160, 16, 2), (33, 1024, 2080, 16, 4),
                                       (3, 2048, 1024, 64, 8), (1, 4096, 4096, 8, 2),
                                       (40, 4224, 1600, 16, 2), (30, 4096, 160, 256, 16),
                                       (4, 4096, 1600, 32, 8), (24, 4160, 1568, 32, 3)])
def test_moe_tiles(T, H, F, E, k, kind):
    Layer(T, H, F, E, k, kind).check()


@pytest.mark.parametrize("T", [2, 12, 40])
def test_moe_unaligned_scales(T):
    layer = Layer(T, 512, 256, 8, 2, "bf16")
    layer.check(odd_scales=True)
    assert torch.equal(layer.run(), layer.run(odd_scales=True))


@pytest.mark.parametrize("T,E", [(20, 64), (64, 32), (64, 6)])
def test_moe_one_expert_of_most_tokens(T, E):
    """More tokens on one expert than are taken at a time."""
    layer = Layer(T, 256, 128, E, 2, "bf16")
    layer.bias[E // 2] += 8.0
    layer.check()


@pytest.mark.parametrize("T", [1, 6, 30])
def test_moe_workspace_is_left_to_itself(T):
    """Other inputs through the same workspace, and the first ones again."""
    layer = Layer(T, 256, 160, 24, 4, "bf16")
    first, x = layer.run(), layer.x
    for seed in range(4):
        layer.x = Layer(T, 256, 160, 24, 4, "bf16", seed + 1).x
        layer.check()
    layer.x = x
    for _ in range(10):
        assert torch.equal(layer.run(), first)


# ------------------------------------------------------------ all of them together

def test_example_layer():
    """examples/mx_layer.py: norm, product, norm and experts, captured and
    replayed.  bf16 outputs are off by at most 2^-9 of each value, and by less
    in the norm; a choice of experts that fp32 logits take differently than 64
    bits is not among these few tokens."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "mx_layer.py")
    spec = importlib.util.spec_from_file_location("mx_layer", path)
    mx_layer = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mx_layer)
    torch.manual_seed(5)
    for error, product in mx_layer.main(["--tokens", "1", "5", "24", "--dim", "512", "--ffn", "256",
                                         "--experts", "12", "--top-k", "3"]):
        assert error <= 2.0 ** -8 and product <= 2.0 ** -8


@pytest.mark.parametrize("rows", [(1 << 22) - 1, 1 << 22, (1 << 26) + 9])
def test_more_rows_than_a_grid(rows):
    """Short rows beyond what one grid holds, and byte offsets beyond 32 bits:
    every row as a call on a few rows of its own has it."""
    K, t = 32, torch.bfloat16
    x = torch.randn(rows, K, generator=gen("rows", rows), device=DEV, dtype=t)
    w = torch.randn(K, generator=gen("weight"), device=DEV, dtype=t)
    c = torch.full((rows, K), 255, device=DEV, dtype=torch.uint8)
    s = torch.full((rows, 1), 77, device=DEV, dtype=torch.uint8)
    picks = [(0, 64), (rows - 64, rows)]
    picks += [(b - 64, min(b + 64, rows)) for b in range((1 << 22) - 1, rows, (1 << 22) - 1)]
    for op in ("norm", "quantize"):
        run = ((lambda a, n, c, s: binding.mx_rmsnorm(a, None, w, 1e-6, n, K, "fp8", None, None, c, s))
               if op == "norm" else (lambda a, n, c, s: binding.mx_quantize(a, n, K, "fp8", c, s)))
        c.fill_(255), s.fill_(77)
        run(x, rows, c, s)
        for lo, hi in picks:
            few_c, few_s = torch.empty_like(c[lo:hi]), torch.empty_like(s[lo:hi])
            run(x[lo:hi].contiguous(), hi - lo, few_c, few_s)
            assert torch.equal(c[lo:hi], few_c) and torch.equal(s[lo:hi], few_s), (op, lo, hi)
        assert not bool((s == 77).any()), op  # every row written (2^-50 is no scale of these)
