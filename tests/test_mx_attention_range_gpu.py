"""Attention over the quantised cache near the ends of fp32's range: values and
scores that are finite, and give finite results.

Bounds are those of test_mx_attention_gpu.py, and for the weights' operands, fp16
whose subnormals are of 2^-24 beside a largest weight of at least 2^10, half a
step of those: 2^-35 of the largest weight, or the weight itself where it is less.
"""
import numpy as np
import pytest
import torch

from oracle import mx
from test_mx_attention_gpu import TYPES, U, Batch, host, put, rounding

pytestmark = pytest.mark.gpu

WIDE = ["bf16", "fp32"]  # fp16 ends at 2^16
# With so many sequences none has its keys cut into shares: a wave (few rows) or a
# workgroup takes them one after the other.
IN_ONE = [(0, 0)] * 600


def values(b, i, array, x):
    """x [keys][heads][head_dim] as sequence i's keys (0) or values (2)."""
    assert x.shape == (len(b.slots[i]), b.Hk, b.D)
    b.pool.put(array, b.slots[i], *mx.quantize(x, b.fmt))


def reference(q, k, v, scale, sees):
    """(y, sum of the weights' shares of |v|, of |v| by 2^-35 or the weight, the
    largest score, the largest sum of |q||k|) in 64 bits."""
    y, mass, low = (np.zeros(q.shape) for _ in range(3))
    top, size = np.zeros(len(q)), np.zeros(len(q))
    for r in range(len(q)):
        j = np.nonzero(sees[r])[0]
        if not len(j):
            continue
        x = (k[j] @ q[r]) * scale
        w = np.exp(x - x.max())
        w /= w.sum()
        y[r], mass[r] = w @ v[j], w @ np.abs(v[j])
        low[r] = np.minimum(w, 2.0 ** -35) @ np.abs(v[j])
        top[r], size[r] = np.abs(x).max(), (np.abs(k[j]) @ np.abs(q[r])).max() * abs(scale)
    return y, mass, low, top, size


def check(b, y, causal=True, window=0, hidden=(), tokens=None):
    """Sequence 0's tokens (all, or those given)."""
    nq, nk = b.seqs[0]
    tokens = np.arange(nq) if tokens is None else np.asarray(tokens)
    a = int(b.starts[0])
    y = host(y).reshape(b.T, b.Hk, b.G, b.D)
    sees = b.sees(0, causal, window, hidden)[tokens].repeat(b.G, 0)
    k, v = b.pool.values(0, b.slots[0]), b.pool.values(2, b.slots[0])
    w = U if b.kind == "fp32" else 2.0 ** -11
    for h in range(b.Hk):
        rows = b.held[a + tokens].reshape(-1, b.Hk, b.G, b.D)[:, h].reshape(-1, b.D)
        seen = sees.any(0)  # what no row sees may be anything
        want, mass, low, top, size = reference(rows, k[seen, h], v[seen, h], b.scale, sees[:, seen])
        off = ((b.D / 4 + 17) * size + 8 * top + 8) * U
        rest = mass * (w + 2 * off[:, None] + (nk / 8 + 64) * U) + low
        got = y[a + tokens, h].reshape(-1, b.D)
        assert np.isfinite(want).all() and np.isfinite(got).all(), (h, np.argwhere(~np.isfinite(got))[:5])
        bad = np.abs(got - want) > rounding(b.kind, np.abs(want) + rest) + rest
        assert not bad.any(), (h, np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


# one token and chunks, in one share of keys and in several
SHAPES = [([(1, 64)], 4), ([(1, 4096)], 4), ([(4, 1024)], 2), ([(40, 256)], 2), ([(40, 4096)], 2)]


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", WIDE)
@pytest.mark.parametrize("seqs,G", SHAPES)
def test_values_near_the_largest(seqs, G, kind, fmt):
    """Values to 2^127: their sums times the weights are beyond fp32, their mean is
    not."""
    b = Batch(seqs, 2, G, 64, 16, fmt, kind)
    nk = seqs[0][1]
    values(b, 0, 2, b.g.uniform(0.5, 1.0, (nk, 2, 64)) * b.g.choice([-1, 1, 1, 1], (nk, 2, 64)) * 2.0 ** 127)
    b.pool.upload()
    check(b, b.run(causal=False), causal=False, tokens=[0, seqs[0][0] // 2, seqs[0][0] - 1])


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", WIDE)
@pytest.mark.parametrize("power", [20, 40, 60, 100, 120])
@pytest.mark.parametrize("seqs,G", [([(1, 1536)], 4), ([(3, 1536)], 4), ([(40, 1536)], 2)])
def test_large_values_before_small_ones(seqs, G, power, kind, fmt):
    """Keys of large values, then of none (zeros; pages of no keys), then of
    ordinary ones, all weights alike: the sums are the large ones'."""
    b = Batch(seqs + IN_ONE, 2, G, 64, 16, fmt, kind)
    run = np.arange(1536) // 512
    x = b.g.uniform(0.5, 1.0, (1536, 2, 64))
    values(b, 0, 2, x * np.array([2.0 ** power, 0.0, 1.0])[run][:, None, None])
    b.pool.upload()
    b.scale = 2.0 ** -30
    tokens = [0, seqs[0][0] - 1]
    check(b, b.run(causal=False), causal=False, tokens=tokens)
    b.table[0, 32:64] = -1
    check(b, b.run(causal=False), causal=False, hidden=np.nonzero(run == 1)[0], tokens=tokens)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", WIDE)
@pytest.mark.parametrize("power", [40, 100, 120])
@pytest.mark.parametrize("seqs", [[(1, 1024)], [(2, 1024)], [(40, 1024)]])
def test_heads_that_prefer_large_and_small_values(seqs, power, kind, fmt):
    """Two heads of a group: the large values, which come first, are all of one's
    result and have no weight, 2^-216, in the other's, which keeps its bits."""
    b = Batch(seqs + IN_ONE, 2, 2, 64, 16, fmt, kind)
    run = (np.arange(1024) // 512)[:, None, None]
    values(b, 0, 0, np.where(run == 0, -4.0, 4.0) * np.ones((1024, 2, 64)))
    values(b, 0, 2, b.g.standard_normal((1024, 2, 64)) * np.where(run == 0, 2.0 ** power, 1.0))
    b.pool.upload()
    b.q, b.held = put(np.broadcast_to(np.array([1.0, -1.0, 1.0, -1.0])[:, None], (b.T, 4, 64)), kind)
    b.scale = 75 / 256
    check(b, b.run(causal=False), causal=False, tokens=[0, seqs[0][0] - 1])


CHUNKS = [([(4, 70)], 1), ([(4, 70)], 4), ([(2, 3000)], 4), ([(40, 200)], 2), ([(70, 1500)], 3)]


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", WIDE)
@pytest.mark.parametrize("power", [20, 60, 112, 120])
@pytest.mark.parametrize("others", [0.0, 1.0])
@pytest.mark.parametrize("seqs,G", CHUNKS)
def test_large_values_that_the_last_token_sees(seqs, G, others, power, kind, fmt):
    """A chunk's last key has large values; all others ordinary ones, or zeros.
    The tokens before it see nothing of them."""
    b = Batch(seqs + (IN_ONE if others else []), 2, G, 64, 16, fmt, kind)
    nq, nk = seqs[0]
    x = b.g.standard_normal((nk, 2, 64)) * others
    x[-1] = b.g.uniform(0.5, 1.0, (2, 64)) * 2.0 ** power
    values(b, 0, 2, x)
    b.pool.upload()
    check(b, b.run(), tokens=sorted({0, nq // 2, nq - 2, nq - 1}))


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", WIDE)
@pytest.mark.parametrize("power", [20, 60, 112, 120])
@pytest.mark.parametrize("others", [[], IN_ONE], ids=["shares", "one"])
@pytest.mark.parametrize("seqs,G", [([(4, 700)], 4), ([(2, 700)], 1), ([(40, 700)], 2)])
def test_large_values_at_the_windows_edge(seqs, G, others, power, kind, fmt):
    """The first key of the first token's window has large values: later tokens do
    not see it, and keep the bits of all keys behind it."""
    b = Batch(seqs + others, 2, G, 64, 16, fmt, kind)
    nq, nk = seqs[0]
    window = 500
    x = b.g.standard_normal((nk, 2, 64))
    x[nk - nq - window + 1] *= 2.0 ** power
    values(b, 0, 2, x)
    b.pool.upload()
    check(b, b.run(window=window), window=window, tokens=sorted({0, 1, nq // 2, nq - 1}))


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("seqs,G", CHUNKS)
def test_blocks_beyond_fp32_where_only_the_last_token_looks(seqs, G, kind, fmt):
    """The largest codes under the largest scale, 448 (6) times 2^127, are no value
    of fp32; the tokens before the last have nothing to do with them."""
    b = Batch(seqs, 2, G, 64, 16, fmt, kind)
    nq, nk = seqs[0]
    last = b.slots[0][-1:]
    code = 0x7E if fmt == "fp8" else 0x77
    b.pool.put(2, last, np.full((1, 2, b.pool.arrays[2].shape[-1]), code, np.uint8),
               np.full((1, 2, 2), 254, np.uint8))
    b.pool.upload()
    check(b, b.run(), tokens=sorted({0, (nq - 1) // 2, nq - 2}))


SCORES = [([(1, 300)], 4), ([(3, 300)], 2), ([(40, 300)], 2)]


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", WIDE)
@pytest.mark.parametrize("seqs,G", SCORES)
def test_small_queries_of_large_keys(seqs, G, kind, fmt):
    """Queries of 2^-124 and keys of 2^126: scores of some ones."""
    b = Batch(seqs, 2, G, 64, 16, fmt, kind)
    x = b.g.uniform(0.5, 1.0, (300, 2, 64)) * b.g.choice([-1, 1], (300, 2, 64))
    values(b, 0, 0, x * 2.0 ** 126)
    b.pool.upload()
    q = b.g.uniform(0.5, 1.0, b.held.shape) * b.g.choice([-1, 1], b.held.shape)
    b.q, b.held = put(q * 2.0 ** -124, kind)
    b.scale = 0.25
    check(b, b.run())


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", WIDE)
@pytest.mark.parametrize("seqs,G", SCORES)
def test_large_queries_across_large_keys(seqs, G, kind, fmt):
    """Queries and keys of 2^100 in different dims: all scores are 0."""
    b = Batch(seqs, 2, G, 64, 16, fmt, kind)
    x = b.g.uniform(0.5, 1.0, (300, 2, 64)) * 2.0 ** 100
    x[..., :32] = 0
    values(b, 0, 0, x)
    b.pool.upload()
    q = b.g.uniform(0.5, 1.0, b.held.shape) * 2.0 ** 100
    q[..., 32:] = 0
    b.q, b.held = put(q, kind)
    check(b, b.run())


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", WIDE)
@pytest.mark.parametrize("scale,q,k", [(3e38, -75, -54), (-3e38, -75, -54), (2.0 ** -140, 70, 68)])
@pytest.mark.parametrize("seqs,G", SCORES)
def test_scales_near_fp32s_ends(seqs, G, scale, q, k, kind, fmt):
    """Scales whose binary form, times log2(e), is past fp32's largest or below its
    smallest normal, for queries and keys whose scores are some ones."""
    b = Batch(seqs, 2, G, 64, 16, fmt, kind)
    x = b.g.uniform(0.5, 1.0, (300, 2, 64)) * b.g.choice([-1, 1], (300, 2, 64))
    values(b, 0, 0, x * 2.0 ** k)
    b.pool.upload()
    x = b.g.uniform(0.5, 1.0, b.held.shape) * b.g.choice([-1, 1], b.held.shape)
    b.q, b.held = put(x * 2.0 ** q, kind)
    b.scale = float(np.float32(scale))
    check(b, b.run())


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", WIDE)
@pytest.mark.parametrize("power", [66, 69, 70, 71, 72, 73, 74, 75, 80, 115])
@pytest.mark.parametrize("seqs,G", SCORES)
def test_large_scores(seqs, G, power, kind, fmt):
    """Queries of 2^power and keys of 2^-50: scores about 2^(power - 46), at the upper
    end 2^69, whose next neighbours in fp32 are some units and more apart: each token
    takes the key of the largest."""
    b = Batch(seqs, 2, G, 64, 16, fmt, kind)
    nq, nk = seqs[0]
    x = np.ones((nk, 2, 64))
    x[7] = 1.5   # that all tokens see
    x[-1] = 2.0  # that the last sees
    values(b, 0, 0, x * 2.0 ** -50)
    b.pool.upload()
    b.q, b.held = put(np.full(b.held.shape, 2.0 ** power), kind)
    y = host(b.run())[1:1 + nq].reshape(nq, 2, G, 64)
    v = b.pool.values(2, b.slots[0])
    want = np.where(np.arange(nq)[:, None, None] == nq - 1, v[-1], v[7])[:, :, None]
    # one weight, its sum and their quotient: exact but for two fp32 roundings and y's own
    assert (np.abs(y - want) <= rounding(kind, np.abs(want)) + 2 * U * np.abs(want)).all()


@pytest.mark.parametrize("kind,fmt", [("bf16", "fp8"), ("fp32", "fp4")])
@pytest.mark.parametrize("nq", [1, 20])
def test_large_and_small_values_within_shares(nq, kind, fmt):
    """Runs of 192 keys of 2^120, zeros and ones, some of each in every share of a
    sequence's keys: references fall within shares, and their parts are joined."""
    from q4_packed_weight_amd import binding
    nk, Hk = 12288, 48
    b = Batch([(nq, nk)], Hk, 1, 32, 64, fmt, kind)
    assert binding.mx_attention_workspace_size(b.T, Hk, Hk, 32, 1, b.width, 64, b.most) > 0
    run = np.arange(nk) // 192 % 3
    x = b.g.uniform(0.5, 1.0, (nk, Hk, 32))
    values(b, 0, 2, x * np.array([2.0 ** 120, 0.0, 1.0])[run][:, None, None])
    # heads by threes: the large values alone, none of them, all alike
    side = np.array([-4.0, 4.0, 0.0])[np.arange(Hk) % 3][:, None]
    values(b, 0, 0, np.where(run == 0, -1.0, 1.0)[:, None, None] * side * np.ones((nk, Hk, 32)))
    b.pool.upload()
    b.q, b.held = put(np.ones((b.T, Hk, 32)), kind)
    b.scale = 75 / 128
    check(b, b.run(causal=False), causal=False, tokens=sorted({0, nq - 1}))
