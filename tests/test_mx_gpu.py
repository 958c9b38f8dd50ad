"""The MX operators on the GPU against the float64 oracle (oracle/mx.py),
through the C ABI.

Bounds count roundings: half a step of the output's type, plus 2^-23 (fp32
sums rounded or cut) for each addition that a sum of the kernel's shape makes,
times the sum of the magnitudes it adds.  Quantisation has no bound: codes and
scales are a function of the values and have to be equal.
"""
import numpy as np
import pytest
import torch

from oracle import mx
from q4_packed_weight_amd import binding
from gpu_util import DEV

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
U = 2.0 ** -23


def rng(*seed):
    return np.random.default_rng((77,) + seed)


def half_step(t):
    return torch.finfo(t).eps / 2


def put(a, t=torch.float32):
    """Array to a GPU tensor of type t, and what it holds there."""
    d = torch.from_numpy(np.ascontiguousarray(a)).to(t).to(DEV)
    return d, d.double().cpu().numpy()


def put8(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


GUARD = 64


class Out:
    """An output with guard elements on both sides that have to stay."""

    def __init__(self, shape, t):
        n = int(np.prod(shape))
        self.fill = 0xA5 if t == torch.uint8 else float("nan")
        self.buf = torch.full((n + 2 * GUARD,), self.fill, dtype=t, device=DEV)
        self.t = self.buf[GUARD:GUARD + n].view(shape)

    def get(self):
        torch.cuda.synchronize()
        g = torch.cat([self.buf[:GUARD], self.buf[-GUARD:]])
        ok = (g == 0xA5).all() if self.fill == 0xA5 else g.isnan().all()
        assert bool(ok), "write past the output"
        return (self.t if self.fill == 0xA5 else self.t.double()).cpu().numpy()


def blocks_out(rows, K, fmt):
    return (Out((rows, K // 2 if fmt == "fp4" else K), torch.uint8),
            Out((rows, K // 32), torch.uint8))


def packed(g, rows, K, fmt, spread=3):
    """Random codes (no e4m3 NaN) and scales around 1; as arrays."""
    c = g.integers(0, 256, (rows, K // 2 if fmt == "fp4" else K)).astype(np.uint8)
    if fmt == "fp8":
        c = np.where((c & 127) == 127, c - 1, c).astype(np.uint8)
    s = g.integers(127 - spread - 2, 127 + spread - 2, (rows, K // 32)).astype(np.uint8)
    return c, s


# ------------------------------------------------------------ quantize

def special_rows(K):
    """Rows that hold what quantisation can get wrong."""
    x = rng(1).standard_normal((12, K))
    x[0] = 0
    x[1] = -0.0
    x[2, 5] = np.nan
    x[3, K - 1] = np.inf
    x[4] *= 2.0 ** -130   # below the normals of fp32
    x[5] *= 2.0 ** 120
    x[6] = np.tile([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], K // 8)   # ties of e2m1
    x[7] = np.tile([256.0, 17.0, 19.0, -21.0, 2.0 ** -10, 3 * 2.0 ** -10, 449.0, 511.0], K // 8)
    x[8] = np.float32(2.0) - np.float32(2.0 ** -23)   # largest below a power
    x[9] *= np.exp2(rng(2).integers(-40, 40, K))
    x[10] = 2.0 ** -126
    x[11] = 65504.0
    return x


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,K", [(12, 32), (12, 96), (12, 1056), (1, 32), (3, 4096), (333, 160),
                                    (1, 16384), (70, 8224)])
def test_quantize_equals_the_oracle(rows, K, kind, fmt):
    x = rng(rows, K).standard_normal((rows, K)) * np.exp2(rng(3).integers(-8, 8, K))
    if rows == 12:
        x = special_rows(K)
    d, held = put(x.astype(np.float32), TYPES[kind])
    codes, scales = blocks_out(rows, K, fmt)
    binding.mx_quantize(d, rows, K, fmt, codes.t, scales.t)
    want = mx.quantize(held, fmt)
    assert np.array_equal(scales.get(), want[1])
    assert np.array_equal(codes.get(), want[0])


def test_quantize_past_one_grid():
    """More chunks than one pass of the largest grid covers."""
    rows, K = 9000, 16384
    x = torch.randn(rows, K, device=DEV, dtype=torch.bfloat16)
    codes = torch.empty(rows, K // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(rows, K // 32, dtype=torch.uint8, device=DEV)
    binding.mx_quantize(x, rows, K, "fp4", codes, scales)
    for a in (0, 4097, rows - 2):
        want = mx.quantize(x[a:a + 2].double().cpu().numpy(), "fp4")
        assert np.array_equal(codes[a:a + 2].cpu().numpy(), want[0])
        assert np.array_equal(scales[a:a + 2].cpu().numpy(), want[1])


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", list(TYPES))
def test_dequantize_every_code_and_scale(kind, fmt):
    """Row s: all codes under scale byte s."""
    K = 32 if fmt == "fp4" else 256
    one = np.arange(K) % (16 if fmt == "fp4" else 256)
    codes = np.tile(mx.pack(one.astype(np.uint8), fmt), (256, 1))
    scales = np.tile(np.arange(256, dtype=np.uint8)[:, None], (1, K // 32))
    out = Out((256, K), TYPES[kind])
    binding.mx_dequantize(put8(codes), put8(scales), 256, K, fmt, out.t)
    with np.errstate(over="ignore"):
        exact = torch.from_numpy(mx.dequantize(codes, scales, fmt).astype(np.float32))
    want = exact.to(TYPES[kind]).double().numpy()
    got = out.get()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])


@pytest.mark.parametrize("rows,K", [(1, 32), (7, 1056), (300, 4096)])
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_dequantize_rows_and_unaligned_scales(rows, K, fmt):
    c, s = packed(rng(4, rows, K), rows, K, fmt)
    shifted = torch.zeros(s.size + 1, dtype=torch.uint8, device=DEV)
    shifted[1:] = put8(s).flatten()
    out = Out((rows, K), torch.float32)
    binding.mx_dequantize(put8(c), shifted[1:], rows, K, fmt, out.t)
    assert np.array_equal(out.get(), mx.dequantize(c, s, fmt))


# ------------------------------------------------------------ rmsnorm

def check_blocks(codes, scales, h, slack, fmt):
    """codes and scales stand for h within half a step and `slack` (relative):
    a block whose largest value lies within the slack of a power of two may
    have either scale."""
    amax = np.abs(h).reshape(*h.shape[:-1], -1, 32).max(-1)
    lo, hi = (mx.scale_bytes(amax * (1 + d), fmt) for d in (-slack, slack))
    assert np.all((scales == lo) | (scales == hi))
    p = np.repeat(2.0 ** (scales.astype(np.float64) - 127), 32, -1)
    v = np.clip(h / p, -mx.TOP[fmt], mx.TOP[fmt])
    bits, low = (1, -1) if fmt == "fp4" else (3, -9)
    _, e = np.frexp(np.maximum(np.abs(v), 1e-30))
    half = 2.0 ** np.maximum(e - 1 - bits, low) / 2
    err = np.abs(mx.dequantize(codes, scales, fmt) / p - v)
    assert np.all(err <= half * (1 + 2.0 ** -10) + slack * np.abs(v))


def norm_slack(K):
    """fp32: a lane's sum of squares (up to 32 values, or 8 for each 1024
    chunks of long rows), 6 + 16 additions across lanes and waves, halved by
    the root; root, quotient and three products."""
    return ((max(32, K / 1024) + 24) / 2 + 6) * U


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,K", [(1, 32), (5, 96), (1, 4096), (33, 1056), (3, 8192), (2, 8224),
                                    (4, 16384), (2, 24608), (2, 40960)])
def test_rmsnorm(rows, K, kind, fmt):
    t = TYPES[kind]
    g = rng(5, rows, K)
    x, xh = put(g.standard_normal((rows, K)) * np.exp(0.6 * g.standard_normal(K)), t)
    res, rh = put(3 * g.standard_normal((rows, K)), t)
    w, wh = put(1 + 0.2 * g.standard_normal(K), t)
    r_out, y = Out((rows, K), t), Out((rows, K), t)
    codes, scales = blocks_out(rows, K, fmt)
    binding.mx_rmsnorm(x, res, w, 1e-5, rows, K, fmt, r_out.t, y.t, codes.t, scales.t)
    r = r_out.get()
    assert np.all(np.abs(r - (xh + rh)) <= half_step(t) * (1 + 2.0 ** -12) * np.abs(xh + rh))
    h = mx.rmsnorm(r, wh, np.float32(1e-5))
    e = norm_slack(K)
    tiny = 2.0 ** -25 if kind == "fp16" else 0.0   # half a step of fp16's subnormals
    assert np.all(np.abs(y.get() - h) <= (half_step(t) + e) * np.abs(h) + tiny)
    check_blocks(codes.get(), scales.get(), h, e, fmt)


def test_rmsnorm_parts_may_be_left_out():
    rows, K, t = 5, 1056, torch.bfloat16
    g = rng(6)
    x, _ = put(g.standard_normal((rows, K)), t)
    res, _ = put(g.standard_normal((rows, K)), t)
    w, _ = put(1 + 0.2 * g.standard_normal(K), t)
    full = [torch.empty(rows, K, dtype=t, device=DEV), torch.empty(rows, K, dtype=t, device=DEV),
            *(o.t for o in blocks_out(rows, K, "fp8"))]
    binding.mx_rmsnorm(x, res, w, 1e-6, rows, K, "fp8", *full)
    for keep in range(3):
        part = [torch.zeros_like(f) if (i if i < 3 else 2) == keep else None
                for i, f in enumerate(full)]
        binding.mx_rmsnorm(x, res, w, 1e-6, rows, K, "fp8", *part)
        for p, f in zip(part, full):
            assert p is None or torch.equal(p, f)
    # without a residual the sum is x itself; a residual of zeros gives the same
    a, b = ([torch.empty_like(f) for f in full] for _ in range(2))
    binding.mx_rmsnorm(x, None, w, 1e-6, rows, K, "fp8", *a)
    binding.mx_rmsnorm(x, torch.zeros_like(x), w, 1e-6, rows, K, "fp8", *b)
    assert torch.equal(a[0], x)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("K", [1056, 40960])
@pytest.mark.parametrize("which", [0, 1])
def test_rmsnorm_in_place(K, which):
    """residual_out may be residual or x itself."""
    rows, t = 4, torch.bfloat16
    g = rng(7, K)
    ins = [put(g.standard_normal((rows, K)), t)[0] for _ in range(2)]
    w, _ = put(1 + 0.2 * g.standard_normal(K), t)
    want = [torch.empty(rows, K, dtype=t, device=DEV), None,
            *(o.t for o in blocks_out(rows, K, "fp8"))]
    binding.mx_rmsnorm(*ins, w, 1e-6, rows, K, "fp8", *want)
    got = [torch.empty_like(w_) for w_ in want[2:]]
    binding.mx_rmsnorm(*ins, w, 1e-6, rows, K, "fp8", ins[which], None, *got)
    assert torch.equal(ins[which], want[0])
    assert all(torch.equal(p, q) for p, q in zip(got, want[2:]))


def test_rmsnorm_special_rows():
    """Zeros stay zeros; a NaN or an infinity makes its row NaN blocks; large
    rows whose squares overflow fp32 give zeros, as the formula does in fp32."""
    rows, K = 4, 96
    x = np.zeros((rows, K), np.float32)
    x[1:3] = rng(8).standard_normal((2, K))
    x[1, 4], x[2, 9] = np.nan, np.inf
    x[3] = 1e30
    d, _ = put(x)
    w, _ = put(np.ones(K))
    y, (codes, scales) = Out((rows, K), torch.float32), blocks_out(rows, K, "fp8")
    binding.mx_rmsnorm(d, None, w, 1e-5, rows, K, "fp8", None, y.t, codes.t, scales.t)
    got, s = y.get(), scales.get()
    assert not got[0].any() and not s[0].any()
    assert np.isnan(got[1]).all() and (s[1] == 255).all()
    assert np.isnan(got[2, 9]) and s[2, 0] == 255
    assert not got[3].any() and not s[3].any()


# ------------------------------------------------------------ matmul

def check_matmul(M, K, N, fmt, kind, seed=9):
    g = rng(seed, M, K, N)
    a, w = packed(g, M, K, fmt), packed(g, N, K, "fp4")
    out = Out((M, N), TYPES[kind])
    binding.mxfp4_matmul(put8(a[0]), put8(a[1]), fmt, put8(w[0]), put8(w[1]), M, K, N, out.t)
    ref, size = mx.matmul(mx.dequantize(*a, fmt), mx.dequantize(*w, "fp4"))
    # 8 levels within an instruction, one addition a step, 16 across waves
    bound = half_step(TYPES[kind]) * np.abs(ref) + (K / 128 + 24) * U * size
    if kind != "fp32" and fmt == "fp8":
        # one instruction for 128 positions: 2^-11 of the largest product
        # (header), twice that as steps may be cut elsewhere
        ad, wd = np.abs(mx.dequantize(*a, fmt)), np.abs(mx.dequantize(*w, "fp4"))
        for s in range(0, K, 128):
            bound += 2.0 ** -10 * (ad[:, None, s:s + 128] * wd[None, :, s:s + 128]).max(-1)
    got = out.get()
    assert np.all(np.abs(got - ref) <= bound), np.max(np.abs(got - ref) / bound)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("M,K,N", [
    (1, 32, 1), (1, 64, 17), (1, 96, 16), (2, 128, 33), (1, 4096, 100), (5, 1056, 257),
    (16, 160, 64), (17, 2048, 40), (32, 1024, 31), (33, 416, 130), (64, 4096, 128), (65, 1056, 65),
    (128, 128, 128), (129, 160, 300), (200, 2080, 513), (256, 512, 256), (300, 1056, 1031),
    (511, 256, 127), (1024, 1024, 1024), (1000, 1056, 999)])
def test_matmul(M, K, N, fmt):
    check_matmul(M, K, N, fmt, "fp32")


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("M,K,N", [(1, 4096, 129), (3, 96, 50), (40, 1056, 64), (130, 544, 260),
                                   (520, 1056, 515)])
def test_matmul_rounds_to_its_type(M, K, N, kind):
    check_matmul(M, K, N, "fp8", kind)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("M", [1, 20, 140, 600])
def test_matmul_one_hot_reads_every_weight_exactly(M, fmt):
    """A = one 1 per row: Y holds weights, bit for bit, from every position of
    a row, under every scale."""
    K, N = 416, 272
    g = rng(10, M)
    wc, ws = packed(g, N, K, "fp4", spread=60)
    at = (np.arange(M) * 7 + g.integers(0, K)) % K
    one = np.zeros((M, K))
    one[np.arange(M), at] = 1.0
    ac, as_ = mx.quantize(one, fmt)
    out = Out((M, N), torch.float32)
    binding.mxfp4_matmul(put8(ac), put8(as_), fmt, put8(wc), put8(ws), M, K, N, out.t)
    assert np.array_equal(out.get(), mx.dequantize(wc, ws, "fp4")[:, at].T)


@pytest.mark.parametrize("M", [1, 20, 140, 600])
def test_matmul_nan_blocks_stay_in_their_row(M):
    K, N = 288, 150
    g = rng(11, M)
    a, w = packed(g, M, K, "fp8"), packed(g, N, K, "fp4")
    a[1][M // 2, 8] = 255     # the last block, past the last whole step
    w[1][N // 3, 0] = 255
    out = Out((M, N), torch.float32)
    binding.mxfp4_matmul(put8(a[0]), put8(a[1]), "fp8", put8(w[0]), put8(w[1]), M, K, N, out.t)
    want = np.zeros((M, N), bool)
    want[M // 2] = want[:, N // 3] = True
    assert np.array_equal(np.isnan(out.get()), want)


@pytest.mark.parametrize("M", [1, 24, 150, 700])
def test_matmul_unaligned_scales_and_outputs(M):
    """Scales at odd addresses and an output that starts off 16 bytes."""
    K, N = 1056, 260
    g = rng(12, M)
    a, w = packed(g, M, K, "fp8"), packed(g, N, K, "fp4")
    off = []
    for s in (a[1], w[1]):
        t = torch.zeros(s.size + 3, dtype=torch.uint8, device=DEV)
        t[3:] = put8(s).flatten()
        off.append(t[3:])
    full = torch.full((M * N + 2,), float("nan"), dtype=torch.bfloat16, device=DEV)
    y = full[1:1 + M * N]
    binding.mxfp4_matmul(put8(a[0]), off[0], "fp8", put8(w[0]), off[1], M, K, N, y)
    ref = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    binding.mxfp4_matmul(put8(a[0]), put8(a[1]), "fp8", put8(w[0]), put8(w[1]), M, K, N, ref)
    assert torch.equal(y.view(M, N), ref)
    assert bool(full[[0, -1]].isnan().all())


# ------------------------------------------------------------ moe

class Layer:
    def __init__(self, T, H, F, E, k, kind, seed=13, bias=True, router=None):
        g = rng(seed, T, H, F, E, k)
        t = TYPES[kind]
        self.size, self.kind, self.k = (T, H, F, E, k), kind, k
        self.x, self.xh = put(g.standard_normal((T, H)), t)
        r = 1.5 * g.standard_normal((E, H)) / np.sqrt(H) if router is None else router
        self.r, self.rh = put(r, t)
        self.b, self.bh = put(0.3 * g.standard_normal(E)) if bias else (None, None)
        uc, us = packed(g, E * 2 * F, H, "fp4", 1)
        dc, ds = packed(g, E * H, F, "fp4", 1)
        us, ds = us - int(np.log2(H) / 2), ds - int(np.log2(F) / 2)
        self.up = mx.dequantize(uc, us, "fp4").reshape(E, 2 * F, H)
        self.down = mx.dequantize(dc, ds, "fp4").reshape(E, H, F)
        self.w = [put8(v) for v in (uc, us, dc, ds)]

    def run(self, out=None, workspace=None):
        T, H = self.size[:2]
        y = torch.empty(T, H, dtype=TYPES[self.kind], device=DEV) if out is None else out
        if workspace is None:
            workspace = torch.full((binding.mxfp4_moe_workspace_size(*self.size),), 0xFF,
                                   dtype=torch.uint8, device=DEV)
        binding.mxfp4_moe(self.x, self.r, self.b, *self.w, *self.size, y, workspace)
        return y

    def check(self):
        T, H = self.size[:2]
        out = Out((T, H), TYPES[self.kind])
        self.run(out.t)
        got = out.get()
        ref, err = mx.moe(self.xh, self.rh, self.bh, self.up, self.down, self.k,
                          2.0 ** -24 if self.kind == "fp32" else 2.0 ** -17)
        bound = half_step(TYPES[self.kind]) * np.abs(ref) + err
        if self.kind == "fp16":
            bound = bound + 2.0 ** -25   # half a step of its subnormals
        assert np.isfinite(err).mean() > 0.5
        assert np.all(np.abs(got - ref) <= bound), np.max(np.abs(got - ref) / bound)


SHAPES = [(1, 64, 32, 4, 1), (1, 96, 64, 4, 4), (1, 512, 256, 64, 8), (2, 160, 96, 1, 1),
          (3, 288, 160, 7, 3), (5, 256, 128, 256, 16), (13, 1056, 736, 24, 3), (16, 128, 64, 5, 2),
          (17, 128, 96, 3, 3), (33, 224, 64, 12, 4), (64, 256, 128, 16, 4), (64, 96, 32, 2, 1),
          (50, 64, 64, 200, 6)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T,H,F,E,k", SHAPES)
def test_moe(T, H, F, E, k, kind):
    Layer(T, H, F, E, k, kind).check()


@pytest.mark.parametrize("T,E", [(65, 8), (150, 6), (70, 256)])
def test_moe_more_tokens_than_run_at_once(T, E):
    Layer(T, 96, 64, E, 2, "bf16").check()


def test_moe_without_bias():
    Layer(6, 128, 64, 9, 2, "bf16", bias=False).check()


@pytest.mark.parametrize("T,k", [(1, 3), (20, 3), (3, 1), (40, 8)])
def test_moe_equal_logits_choose_the_lower_index(T, k):
    """A router of zeros: every token takes experts 0 .. k-1 in equal parts."""
    layer = Layer(T, 96, 64, 24, k, "fp32", bias=False, router=np.zeros((24, 96)))
    got = layer.run().double().cpu().numpy()
    want = np.zeros_like(layer.xh)
    for e in range(k):
        gu = layer.xh @ layer.up[e].T
        want += mx.silu(gu[:, :64]) * gu[:, 64:] @ layer.down[e].T / k
    size = np.abs(want).max()
    assert np.all(np.abs(got - want) <= 2.0 ** -15 * size)


@pytest.mark.parametrize("T", [1, 30])
def test_moe_nan_logits_come_last(T):
    """A NaN bias keeps its expert out while k others are there."""
    layer = Layer(T, 96, 64, 6, 3, "fp32")
    layer.b[2] = float("nan")
    layer.bh = layer.bh.copy()
    layer.bh[2] = -1e9
    layer.check()


def test_moe_same_expert_for_every_token():
    """All 64 tokens on one expert of many: full tiles of tokens."""
    layer = Layer(64, 128, 64, 32, 1, "bf16")
    layer.b[5] = 100.0
    layer.bh = layer.b.double().cpu().numpy()
    layer.check()


def test_moe_nan_input_stays_in_its_token():
    layer = Layer(9, 128, 64, 6, 2, "bf16")
    clean = layer.run()
    layer.x[4, 17] = float("nan")
    got = layer.run()
    assert bool(got[4].isnan().all())
    keep = [t for t in range(9) if t != 4]
    assert torch.equal(got[keep], clean[keep])


# ------------------------------------------------------------ all of them

def calls():
    """One call of each operator and its outputs, inputs in place."""
    g = rng(14)
    t = torch.bfloat16
    x, _ = put(g.standard_normal((40, 1056)), t)
    w, _ = put(1 + 0.2 * g.standard_normal(1056), t)
    r, y = torch.empty_like(x), torch.empty_like(x)
    c4, s4 = (o.t for o in blocks_out(40, 1056, "fp4"))
    c8, s8 = (o.t for o in blocks_out(40, 1056, "fp8"))
    out = []
    out.append((lambda: binding.mx_quantize(x, 40, 1056, "fp4", c4, s4), [c4, s4]))
    a = [put8(v) for v in packed(g, 40, 1056, "fp8")]
    b = [put8(v) for v in packed(g, 300, 1056, "fp4")]
    v = torch.empty(40, 1056, dtype=t, device=DEV)
    out.append((lambda: binding.mx_dequantize(*a, 40, 1056, "fp8", v), [v]))
    out.append((lambda: binding.mx_rmsnorm(x, x, w, 1e-5, 40, 1056, "fp8", r, y, c8, s8),
                [r, y, c8, s8]))
    z = torch.empty(40, 300, device=DEV)
    out.append((lambda: binding.mxfp4_matmul(*a, "fp8", *b, 40, 1056, 300, z), [z]))
    big = [put8(q) for q in packed(g, 700, 1056, "fp8")]
    zb = torch.empty(700, 300, device=DEV)
    out.append((lambda: binding.mxfp4_matmul(*big, "fp8", *b, 700, 1056, 300, zb), [zb]))
    for T in (1, 20):
        layer = Layer(T, 160, 96, 12, 3, "bf16")
        ly = torch.empty(T, 160, dtype=t, device=DEV)
        ws = torch.empty(binding.mxfp4_moe_workspace_size(*layer.size), dtype=torch.uint8,
                         device=DEV)
        out.append((lambda layer=layer, ly=ly, ws=ws: layer.run(ly, ws), [ly]))
    return out


def bits(tensors):
    torch.cuda.synchronize()
    return [t.view(torch.uint8).cpu() for t in tensors]


def clear(tensors):
    for t in tensors:
        t.fill_(0x5A if t.dtype == torch.uint8 else float("nan"))


def test_repeatable_on_another_stream():
    """The same bits again, on a stream of its own."""
    s = torch.cuda.Stream()
    for call, outs in calls():
        call()
        first = bits(outs)
        clear(outs)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            call()
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(a, b) for a, b in zip(first, bits(outs)))


def test_graph_replays():
    """Captured, and replayed with eager work between: the eager bits each time."""
    for call, outs in calls():
        call()
        eager = bits(outs)
        g = torch.cuda.CUDAGraph()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
            call()
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        for _ in range(4):
            clear(outs)
            torch.cuda.synchronize()
            g.replay()
            assert all(torch.equal(a, b) for a, b in zip(eager, bits(outs)))
