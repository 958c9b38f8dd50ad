"""Rotary positions, the quantised cache and attention over it on the GPU,
against the float64 oracle (oracle/mx.py), through the C ABI.

Bounds count roundings (U = 2^-23, an fp32 rounding or cut):
  rotary     half a step of the type; the angle's part of a turn, held in fp32,
             is off by 2^-26 of a turn (under 4e-7 of an angle in all, with its
             cosine's own two steps under 5 U), and three more roundings
  cache      none: codes and scales are a function of the values
  attention  half a step of the type, and of what the weights share of |v|
               2^-11 (bf16, fp16) or U (fp32) for a weight's rounding (fp16 has
               11 bits: half a step is up to 2^-11 of the value; a second fp16
               holds what is left, under 2^(e-11), to half a step of 2^(e-23)),
               twice what a score is off by (numerator and denominator): an fp32
               sum of head_dim products, up to head_dim / 4 + 17 additions of U
               of the sum of magnitudes, and 8 U of the score and 8 U for the
               exponential,
               one U for each of the additions in a chain: a wave's eighth of
               the keys, 64 for the joins
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
FILL = 31.0  # of rows that have to stay


def rng(*seed):
    return np.random.default_rng((123,) + tuple(int(s) for s in seed))


def rounding(kind, size):
    """Half a step at values up to `size`: relative, and no less than half of the
    step of the type's subnormals (fp16: 2^-24)."""
    t = torch.finfo(TYPES[kind])
    return np.maximum(t.eps / 2 * size, t.smallest_normal * t.eps / 2)


def put(a, kind):
    """Array to a GPU tensor, and what it holds there."""
    d = torch.from_numpy(np.ascontiguousarray(a)).to(TYPES[kind]).to(DEV)
    return d, d.double().cpu().numpy()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy()


# ------------------------------------------------------------ rotary

def rotary_bound(want, x, amplitude, R, layout, kind):
    h = R // 2
    one = slice(0, h) if layout == "half" else slice(0, R, 2)
    two = slice(h, R) if layout == "half" else slice(1, R, 2)
    size = np.zeros_like(want)
    size[..., one] = size[..., two] = np.abs(x[..., one]) + np.abs(x[..., two])
    rest = 8 * U * amplitude * size
    return rounding(kind, np.abs(want) + rest) + rest


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T,H,D,R,extra", [(1, 40, 128, 128, 0), (1, 1, 8, 2, 8), (333, 5, 96, 64, 96),
                                           (7, 3, 64, 64, 8), (5, 13, 80, 50, 0), (64, 2, 256, 16, 0),
                                           (1030, 6, 128, 32, 256), (3, 2, 512, 512, 0),
                                           (300, 1, 32, 2, 0), (9, 130, 64, 48, 0)])
def test_rotary(T, H, D, R, extra, kind, layout):
    g = rng(T, H, D, R)
    wide = g.standard_normal((T, H * D + extra)) * 3
    d, held = put(wide, kind)
    x = held[:, :H * D].reshape(T, H, D)
    pos = g.integers(0, 1 << 20, T)
    pos[0] = (1 << 20) + 7
    f, _ = binding.mx_rotary_frequencies(R, 10000.0, "yarn", 4.0)
    amp = 1.25
    y = torch.full((T + 2, H * D), FILL, dtype=TYPES[kind], device=DEV)
    binding.mx_rotary(d[:, :H * D], dev(pos), f.to(DEV), amp, T, H, D, R, layout, y[1:T + 1])
    want = mx.rotary(x, pos, f.numpy(), amp, R, layout)
    got = host(y)
    assert (got[0] == FILL).all() and (got[-1] == FILL).all()
    got = got[1:-1].reshape(T, H, D)
    assert (np.abs(got - want) <= rotary_bound(want, x, amp, R, layout, kind)).all()
    # in place, in a wider row: the same bits, the rest of the row untouched
    binding.mx_rotary(d[:, :H * D], dev(pos), f.to(DEV), amp, T, H, D, R, layout, d[:, :H * D])
    after = host(d)
    assert np.array_equal(after[:, :H * D].reshape(T, H, D), got)
    assert np.array_equal(after[:, H * D:], held[:, H * D:])


def test_rotary_of_far_and_negative_positions():
    """Angles of 10^9 radians: 32 bits would hold none of them."""
    pos = np.array([0, 1, -1, 1 << 30, -(1 << 30), 999999937])
    x = rng(5).standard_normal((6, 2, 64))
    d, held = put(x, "fp32")
    f, _ = binding.mx_rotary_frequencies(64)
    y = torch.empty_like(d)
    binding.mx_rotary(d, dev(pos), f.to(DEV), 1.0, 6, 2, 64, 64, "half", y)
    want = mx.rotary(held, pos, f.numpy(), 1.0, 64, "half")
    # fp64: a product of 2^30, rounded twice, in radians
    far = 2.0 ** 30 * 2.0 ** -52
    bound = rotary_bound(want, held, 1.0, 64, "half", "fp32") + far * 8
    assert (np.abs(host(y) - want) <= bound).all()
    assert np.array_equal(host(y)[0], held[0])  # an angle of zero


def test_rotary_keeps_what_is_not_finite_to_its_pair():
    d, _ = put(np.ones((1, 1, 64)), "bf16")
    d[0, 0, 3] = float("nan")
    d[0, 0, 60] = float("inf")
    f, _ = binding.mx_rotary_frequencies(32)
    y = torch.empty_like(d)
    binding.mx_rotary(d, dev(np.array([5])), f.to(DEV), 1.0, 1, 1, 64, 32, "half", y)
    bad = ~np.isfinite(host(y)[0, 0])
    assert np.nonzero(bad)[0].tolist() == [3, 19, 60]


# ------------------------------------------------------------ cache

class Pool:
    """Pages of random bytes, e4m3 NaN and NaN blocks among them."""

    def __init__(self, pages, heads, size, D, fmt, seed=1):
        g = rng(pages, heads, size, D, seed)
        self.fmt, self.shape = fmt, (pages, heads, size)
        n = D if fmt == "fp8" else D // 2
        self.arrays = []
        for _ in range(2):
            self.arrays.append(g.integers(0, 256, (pages, heads, size, n)).astype(np.uint8))
            self.arrays.append(g.choice(np.array([0, 120, 127, 254, 255], np.uint8),
                                        (pages, heads, size, D // 32)))
        self.upload()

    def upload(self):
        self.t = [dev(a) for a in self.arrays]

    def download(self):
        torch.cuda.synchronize()
        return [t.cpu().numpy() for t in self.t]

    def put(self, i, slots, codes, scales):
        """Rows [tokens][heads][..] into arrays i and i + 1."""
        page, place = slots // self.shape[2], slots % self.shape[2]
        self.arrays[i][page, :, place] = codes
        self.arrays[i + 1][page, :, place] = scales

    def values(self, i, slots):
        if not len(slots):
            return np.zeros((0, self.shape[1], self.arrays[i + 1].shape[-1] * 32))
        page, place = slots // self.shape[2], slots % self.shape[2]
        with np.errstate(invalid="ignore"):
            return mx.dequantize(self.arrays[i][page, :, place], self.arrays[i + 1][page, :, place],
                                 self.fmt)


CACHES = [(1, 1, 32, 16, 3), (64, 8, 128, 16, 20), (333, 5, 96, 64, 7), (17, 3, 256, 1, 40),
          (50, 2, 64, 7, 9), (9, 40, 160, 256, 2)]


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T,H,D,size,pages", CACHES)
def test_cache_write(T, H, D, size, pages, kind, fmt):
    g = rng(T, H, D, size)
    pool = Pool(pages, H, size, D, fmt)
    slots = g.permutation(pages * size)[:T].astype(np.int64)
    assert len(slots) == T
    left_out = g.random(T) < 0.2
    rows = g.standard_normal((2, T, H, D)) * np.exp2(g.integers(-6, 6, (2, T, H, D)))
    rows[0, -1, 0, 5], rows[1, 0, -1, 3] = np.nan, np.inf
    kd, k = put(rows[0], kind)
    wide, v = put(np.concatenate([rows[1].reshape(T, -1), rows[0].reshape(T, -1)], 1), kind)
    v = v[:, :H * D].reshape(T, H, D)
    for i, x in ((0, k), (2, v)):
        c, s = mx.quantize(x, fmt)
        pool.put(i, slots[~left_out], c[~left_out], s[~left_out])
    sent = np.where(left_out, g.choice([-1, -5, pages * size, 1 << 40], T), slots)
    other = Pool(pages, H, size, D, fmt)
    binding.mx_cache_write(kd, wide[:, :H * D], dev(sent), T, H, D, fmt, *other.t, pages, size)
    for a, b in zip(other.download(), pool.arrays):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T,H,D,size,pages", CACHES)
def test_cache_read(T, H, D, size, pages, kind, fmt):
    g = rng(T, H, D, size, 2)
    pool = Pool(pages, H, size, D, fmt)
    for i in (1, 3):  # powers that every type holds, and NaN
        pool.arrays[i] = g.choice(np.array([119, 120, 121, 127, 255], np.uint8), pool.arrays[i].shape)
    pool.upload()
    slots = g.integers(0, pages * size, T)  # some more than once
    sent = np.where(g.random(T) < 0.2, g.choice([-1, pages * size, -(1 << 50)], T), slots)
    gone = sent != slots
    k = torch.full((T + 2, H * D), FILL, dtype=TYPES[kind], device=DEV)
    v = torch.full((T, 2 * H * D), FILL, dtype=TYPES[kind], device=DEV)
    binding.mx_cache_read(dev(sent), T, H, D, fmt, *pool.t, pages, size, k[1:-1], v[:, H * D:])
    for got, i in ((host(k)[1:-1], 0), (host(v)[:, H * D:], 2)):
        want = np.where(gone[:, None, None], 0, pool.values(i, slots)).reshape(T, -1)
        want = torch.from_numpy(want).to(TYPES[kind]).double().numpy()
        assert np.array_equal(got, want, equal_nan=True)
    assert (host(k)[[0, -1]] == FILL).all() and (host(v)[:, :H * D] == FILL).all()


def test_cache_rows_past_32_bit_offsets():
    """A pool of more than 4 GiB of codes: its last page, written and read back,
    and seen by attention."""
    H, D, size = 64, 256, 4096
    pages = (5 << 30) // (H * D * size)
    n = pages * size
    k_codes = torch.zeros(pages, H, size, D, dtype=torch.uint8, device=DEV)
    v_codes = torch.zeros_like(k_codes)
    k_scales, v_scales = (torch.zeros(pages, H, size, D // 32, dtype=torch.uint8, device=DEV)
                          for _ in range(2))
    pool = k_codes, k_scales, v_codes, v_scales
    g = rng(9)
    T = 40
    slots = np.arange(n - T, n)
    kd, k = put(g.standard_normal((T, H, D)), "bf16")
    vd, v = put(g.standard_normal((T, H, D)), "bf16")
    binding.mx_cache_write(kd, vd, dev(slots), T, H, D, "fp8", *pool, pages, size)
    ko, vo = torch.empty_like(kd), torch.empty_like(vd)
    binding.mx_cache_read(dev(slots), T, H, D, "fp8", *pool, pages, size, ko, vo)
    k, v = (mx.dequantize(*mx.quantize(x, "fp8"), "fp8") for x in (k, v))
    assert np.array_equal(host(ko), k) and np.array_equal(host(vo), v)
    assert not k_codes.view(-1)[:1 << 32].any() and not v_codes.view(-1)[:1 << 32].any()
    q = torch.zeros(1, H, D, dtype=torch.bfloat16, device=DEV)  # the mean of the values
    y = torch.empty_like(q)
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device=DEV)
    starts, counts = (torch.tensor(a, dtype=torch.int32, device=DEV) for a in ([0, 1], [size]))
    ws = workspace(1, H, H, D, 1, 1, size, 1)
    binding.mx_attention(q, starts, counts, table, 1, H, H, D, 1, 1, 1, 1.0, True, T, "fp8", *pool,
                         pages, size, y, ws)
    want = v.mean(0)
    # bf16 holds 8 bits: half a step is up to 2^-8 of the value; equal weights have one share each
    bad = np.abs(host(y)[0] - want) > 2.0 ** -8 * np.abs(want) + 2.0 ** -11 * np.abs(v).mean(0)
    assert not bad.any(), np.argwhere(bad)[:5]


# ------------------------------------------------------------ attention

def workspace(*sizes):
    n = binding.mx_attention_workspace_size(*sizes)
    return torch.full((n,), 0xA7, dtype=torch.uint8, device=DEV)


class Batch:
    """Sequences of (new tokens, keys) over a pool of shuffled pages; places
    behind a sequence's keys and pages of none hold random bytes."""

    def __init__(self, seqs, Hk, G, D, size, fmt, kind, seed=0, sharp=1.0, before=1, after=2,
                 extra=0):
        g = rng(len(seqs), Hk, G, D, size, seed, *[a for s in seqs for a in s])
        self.g, self.seqs, self.Hk, self.G, self.D, self.size = g, seqs, Hk, G, D, size
        self.fmt, self.kind = fmt, kind
        need = [-(-nk // size) for _, nk in seqs]
        self.width = max(max(need) + extra, 1)
        self.n_pages = sum(need) + 3
        self.pool = Pool(self.n_pages, Hk, size, D, fmt, seed)
        order = g.permutation(self.n_pages)
        self.table = g.choice(np.array([-1, self.n_pages, 1 << 30, 0]), (len(seqs), self.width))
        self.slots = []
        at = 0
        for i, (n, (_, nk)) in enumerate(zip(need, seqs)):
            self.table[i, :n] = order[at:at + n]
            at += n
            j = np.arange(nk)
            self.slots.append(self.table[i, j // size] * size + j % size)
            spread = np.exp(0.5 * g.standard_normal((2, Hk, D)))
            for a in range(2 if nk else 0):
                x = g.standard_normal((nk, Hk, D)) * spread[a]
                self.pool.put(2 * a, self.slots[i], *mx.quantize(x, fmt))
        self.pool.upload()
        starts = np.cumsum([before] + [nq for nq, _ in seqs])
        self.starts, self.T = starts, int(starts[-1]) + after
        self.counts = np.array([nk for _, nk in seqs])
        self.most = max(max(nq for nq, _ in seqs), 1)
        q = g.standard_normal((self.T, Hk * G, D)) * sharp
        self.q, self.held = put(q, kind)
        self.scale = D ** -0.5

    def run(self, causal=True, window=0, y=None, ws=None, most=None):
        H, t = self.Hk * self.G, torch.int32
        most = most or self.most
        if y is None:
            y = torch.full((self.T, H * self.D), FILL, dtype=TYPES[self.kind], device=DEV)
        sizes = self.T, H, self.Hk, self.D, len(self.seqs), self.width, self.size, most
        if ws is None:
            ws = workspace(*sizes)
        args = [dev(a).to(t) for a in (self.starts, self.counts, self.table)]
        binding.mx_attention(self.q, *args, self.T, H, self.Hk, self.D, len(self.seqs), self.width,
                             most, self.scale, causal, window, self.fmt, *self.pool.t,
                             self.n_pages, self.size, y, ws)
        return y

    def sees(self, i, causal, window, hidden=()):
        """[tokens][keys] of sequence i."""
        nq, nk = self.seqs[i]
        j, t = np.arange(nk), np.arange(nq)[:, None]
        last = nk - nq + t if causal else np.full((nq, 1), nk - 1)
        s = j <= last
        if window:
            s &= j > last - window
        if len(hidden):
            s[:, np.asarray(hidden)] = False
        return s

    def check(self, y, causal=True, window=0, hidden={}, most=None, sample=None):
        y = host(y).reshape(self.T, self.Hk, self.G, self.D)
        untouched = np.ones(self.T, bool)
        w = U if self.kind == "fp32" else 2.0 ** -11
        for i, (nq, nk) in enumerate(self.seqs):
            a = int(self.starts[i])
            n = min(nq, most or nq)
            untouched[a:a + n] = False
            tokens = np.arange(n) if sample is None or n <= sample else np.unique(
                np.r_[0, n - 1, self.g.integers(0, n, sample)])
            sees = self.sees(i, causal, window, hidden.get(i, ()))[tokens].repeat(self.G, 0)
            k, v = self.pool.values(0, self.slots[i]), self.pool.values(2, self.slots[i])
            for h in range(self.Hk):
                rows = self.held[a + tokens].reshape(-1, self.Hk, self.G, self.D)[:, h].reshape(-1, self.D)
                want, mass, top, size = mx.attention(rows, k[:, h], v[:, h], self.scale, sees)
                off = ((self.D / 4 + 17) * size + 8 * top + 8) * U
                rest = mass * (w + 2 * off[:, None] + (nk / 8 + 64) * U)
                bound = rounding(self.kind, np.abs(want) + rest) + rest
                got = y[a + tokens, h].reshape(-1, self.D)
                nan = np.isnan(want)
                assert np.array_equal(np.isnan(got), nan), (i, h)
                bad = ~(np.abs(got - want) <= bound) & ~nan
                assert not bad.any(), (i, h, np.argwhere(bad)[:5], np.abs(got - want)[bad].max())
        assert (y[untouched] == FILL).all()


SEQS = [[(1, 1)], [(1, 1000)], [(1, 33), (1, 0), (1, 512), (0, 40), (1, 64)],
        [(5, 5), (1, 300), (17, 90), (0, 0), (3, 1)], [(40, 203)]]


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("seqs", SEQS, ids=range(len(SEQS)))
@pytest.mark.parametrize("Hk,G,D,size", [(2, 4, 128, 16), (1, 1, 32, 1), (3, 7, 96, 32),
                                         (2, 16, 64, 64), (1, 5, 256, 7), (2, 2, 160, 256)])
def test_attention(Hk, G, D, size, seqs, kind, fmt):
    b = Batch(seqs, Hk, G, D, size, fmt, kind, sharp=2.0)
    b.check(b.run())


@pytest.mark.parametrize("kind,fmt", [("bf16", "fp8"), ("fp32", "fp4"), ("fp16", "fp8")])
@pytest.mark.parametrize("window", [1, 2, 31, 64, 1000])
def test_attention_window(window, kind, fmt):
    b = Batch([(1, 700), (37, 300), (2, 2), (70, 70), (130, 4)], 2, 3, 64, 16, fmt, kind)
    b.check(b.run(window=window), window=window)


@pytest.mark.parametrize("kind,fmt", [("bf16", "fp4"), ("fp32", "fp8"), ("fp16", "fp8")])
def test_attention_without_causal(kind, fmt):
    b = Batch([(1, 50), (37, 300), (5, 0), (20, 3)], 3, 2, 96, 16, fmt, kind)
    b.check(b.run(causal=False), causal=False)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("seqs,G", [([(1, 5000)], 4), ([(1, 5000), (1, 20), (1, 300)], 16),
                                    ([(9, 3001), (2, 4000)], 2)])
def test_attention_over_ranges_of_keys(seqs, G, kind, fmt):
    """Long sequences next to short ones: the keys cut into ranges and joined."""
    b = Batch(seqs, 2, G, 128, 16, fmt, kind, sharp=3.0)
    assert binding.mx_attention_workspace_size(b.T, 2 * G, 2, 128, len(seqs), b.width, 16,
                                               b.most) > 0
    b.check(b.run())
    b.check(b.run(window=900), window=900)


@pytest.mark.parametrize("kind,fmt,G,D", [("bf16", "fp8", 4, 128), ("fp16", "fp4", 3, 96),
                                          ("fp32", "fp8", 1, 64), ("bf16", "fp4", 8, 256)])
def test_attention_of_chunks(kind, fmt, G, D):
    """Chunks of some hundred tokens, a single token and an empty one among them."""
    b = Batch([(300, 1000), (1, 77), (0, 10), (129, 129), (64, 2000)], 2, G, D, 64, fmt, kind,
              sharp=2.0)
    b.check(b.run(), sample=12)
    b.check(b.run(window=100), window=100, sample=12)
    b.check(b.run(causal=False), causal=False, sample=12)


def test_attention_prefers_nothing_it_cannot_see():
    """Huge, infinite and NaN keys and values where no token or only later ones
    look: block 255 and the e4m3 NaN, in the keys' own pages."""
    for fmt in ("fp4", "fp8"):
        for kind in TYPES:
            for seqs in ([(6, 70)], [(60, 200)], [(1, 45)]):
                b = Batch(seqs, 2, 3, 64, 16, fmt, kind)
                nq, nk = seqs[0]
                last = b.slots[0][nk - 1:]
                for i in (0, 2):
                    shape = (1, 2, 64 if fmt == "fp8" else 32)
                    codes = np.full(shape, 0x7F if fmt == "fp8" else 0x77, np.uint8)
                    b.pool.put(i, last, codes, np.full((1, 2, 2), 240 if i == 0 else 127, np.uint8))
                if nq > 1:  # only the last token sees them: a NaN block of values
                    b.pool.arrays[3][last // 16, :, last % 16, 1] = 255
                b.pool.upload()
                y = host(b.run()).reshape(b.T, 2, 3, 64)[1:1 + nq]
                if fmt == "fp8" or nq > 1:
                    assert np.isnan(y[-1, ..., 32:]).all()
                assert np.isfinite(y[:-1]).all()
                if nq > 1:
                    # all but the last as if the key were not there
                    rows = b.held[1:nq].reshape(-1, 2, 3, 64)
                    sees = b.sees(0, True, 0)[:-1].repeat(3, 0)[:, :-1]
                    for h in range(2):
                        want, mass, top, size = mx.attention(
                            rows[:, h].reshape(-1, 64), b.pool.values(0, b.slots[0][:-1])[:, h],
                            b.pool.values(2, b.slots[0][:-1])[:, h], b.scale, sees)
                        off = ((33 * size + 8 * top + 8) * U)[:, None]
                        rest = mass * (2.0 ** -11 + 2 * off + 100 * U)
                        bound = rounding(kind, np.abs(want) + rest) + rest
                        assert (np.abs(y[:-1, h].reshape(-1, 64) - want) <= bound).all()


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("nq", [1, 40, 150])
def test_attention_nan_reaches_those_that_see_it(nq, fmt):
    """A NaN block of a key: all of the row; of a value: its 32 dims; a query
    that is not finite: its own row."""
    b = Batch([(nq, 400)], 2, 2, 64, 16, fmt, "bf16", after=0, before=0)
    key = 400 - (nq + 1) // 2 - 1
    s = b.slots[0][key]
    b.pool.arrays[3][s // 16, 0, s % 16, 1] = 255  # head 0, dims 32 .. 63
    s2 = b.slots[0][key - 100]
    b.pool.arrays[1][s2 // 16, 1, s2 % 16, 0] = 255  # head 1
    b.q[nq - 1, 1, 7] = float("inf")
    b.held[nq - 1, 1, 7] = np.inf
    b.pool.upload()
    got = np.isnan(host(b.run()).reshape(nq, 2, 2, 64))
    sees = b.sees(0, True, 0)
    want = np.zeros_like(got)
    want[:, 0, :, 32:] = sees[:, key][:, None, None]
    want[:, 1] = sees[:, key - 100][:, None, None]
    want[nq - 1, 0, 1] = True
    assert np.array_equal(got, want)


def test_attention_pages_of_no_keys():
    """Entries outside the pool, within a sequence's keys, hide their page."""
    for seqs in ([(1, 333)], [(50, 333)], [(200, 333), (1, 100)]):
        b = Batch(seqs, 2, 4, 128, 16, "fp8", "bf16")
        for bad in (-1, b.n_pages, 1 << 30, -(1 << 31)):
            b.table[0, 3] = bad
            b.check(b.run(), hidden={0: range(48, 64)}, sample=12)
        b.table[0, :] = -7
        b.check(b.run(), hidden={0: range(333)}, sample=12)


def test_attention_counts_and_starts_out_of_range():
    """Counts above what the pages hold are cut, negative ones are none; tokens
    past max_queries stay."""
    b = Batch([(3, 64), (2, 10), (4, 30)], 1, 4, 64, 16, "fp8", "bf16")
    b.counts = np.array([1 << 30, -5, 30])
    b.seqs = [(3, 64), (2, 0), (4, 30)]
    b.check(b.run())
    b.slots[1] = b.slots[1][:0]
    b.check(b.run(most=3), most=3)


def test_attention_powers_far_apart():
    """Blocks whose scales lie 2^20 apart, and rows of q from 2^-100 to 2^90."""
    for fmt in ("fp4", "fp8"):
        for kind in ("bf16", "fp32"):
            b = Batch([(4, 100), (40, 300)], 2, 2, 64, 16, fmt, kind)
            for i in (0, 1):
                n = len(b.slots[i])
                k = b.g.standard_normal((n, 2, 64)) * np.exp2(b.g.integers(-9, 10, (n, 2, 2))).repeat(32, -1)
                v = b.g.standard_normal((n, 2, 64)) * np.exp2(b.g.integers(-9, 10, (n, 2, 2))).repeat(32, -1)
                b.pool.put(0, b.slots[i], *mx.quantize(k, fmt))
                b.pool.put(2, b.slots[i], *mx.quantize(v, fmt))
            b.pool.upload()
            e = b.g.integers(-100, -6, (b.T, 4, 1))
            b.q, b.held = put(b.held * np.exp2(e), kind)
            b.check(b.run())
            b.q, b.held = put(b.held * np.exp2(90.0), kind)
            b.scale = 2.0 ** -90
            b.check(b.run())


def test_attention_is_the_same_at_each_call():
    """In a graph too, replayed among other work, and with a used workspace."""
    b = Batch([(1, 3000), (1, 50), (1, 4096)], 4, 4, 128, 16, "fp8", "bf16")
    c = Batch([(200, 900), (1, 50)], 4, 4, 128, 16, "fp8", "bf16")
    for x in (b, c):
        ws = workspace(x.T, 16, 4, 128, len(x.seqs), x.width, 16, x.most)
        first = host(x.run(ws=ws))
        assert np.array_equal(host(x.run(ws=ws)), first)
        y = torch.full((x.T, 16 * 128), FILL, dtype=torch.bfloat16, device=DEV)
        args = [dev(a).to(torch.int32) for a in (x.starts, x.counts, x.table)]
        torch.cuda.synchronize()
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
            binding.mx_attention(x.q, *args, x.T, 16, 4, 128, len(x.seqs), x.width, x.most, x.scale,
                                 True, 0, "fp8", *x.pool.t, x.n_pages, 16, y, ws)
        for _ in range(3):
            y.fill_(FILL)
            ws.fill_(0x5A)
            graph.replay()
            assert np.array_equal(host(y), first)
