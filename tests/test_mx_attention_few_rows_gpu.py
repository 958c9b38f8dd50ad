"""Attention of a few tokens over the quantised cache: more than one token, and no
more than 16 pairs of token and head to a key head, where some rows of a step see
keys that others do not.  Bounds as in test_mx_attention_gpu.py."""
import numpy as np
import pytest
import torch

from oracle import mx
from q4_packed_weight_amd import binding
from test_mx_attention_gpu import TYPES, Batch, host, put

pytestmark = pytest.mark.gpu


def batch(seqs, Hk, G, D, size, fmt, kind, **more):
    b = Batch(seqs, Hk, G, D, size, fmt, kind, **more)
    assert 1 < b.most and b.most * G <= 16
    return b


SEQS = [([(2, 70)], 8), ([(4, 4), (1, 300), (3, 33), (0, 9), (2, 1)], 4), ([(16, 16), (5, 203)], 1),
        ([(3, 1025)], 5)]


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("seqs,G", SEQS, ids=range(len(SEQS)))
@pytest.mark.parametrize("D,size", [(32, 1), (64, 16), (96, 32), (128, 16), (160, 7), (256, 64)])
def test_few_rows(D, size, seqs, G, kind, fmt):
    b = batch(seqs, 2, G, D, size, fmt, kind, sharp=2.0)
    b.check(b.run())
    b.check(b.run(window=50), window=50)
    b.check(b.run(causal=False), causal=False)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("seqs,G,D", [([(4, 5000)], 4, 128), ([(2, 4000), (1, 20), (3, 700)], 5, 64),
                                      ([(2, 3000)], 8, 256), ([(7, 2500), (4, 90)], 2, 96)])
def test_few_rows_over_ranges_of_keys(seqs, G, D, kind, fmt):
    b = batch(seqs, 2, G, D, 16, fmt, kind, sharp=3.0)
    assert binding.mx_attention_workspace_size(b.T, 2 * G, 2, D, len(seqs), b.width, 16, b.most) > 0
    b.check(b.run())
    b.check(b.run(window=900), window=900)


@pytest.mark.parametrize("kind,fmt", [("bf16", "fp8"), ("fp16", "fp4"), ("fp32", "fp8")])
@pytest.mark.parametrize("window", [1, 2, 3, 31, 64, 1000])
def test_few_rows_window(window, kind, fmt):
    b = batch([(1, 700), (4, 300), (2, 2), (3, 70), (4, 2), (4, 1500)], 2, 3, 128, 16, fmt, kind)
    b.check(b.run(window=window), window=window)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("seqs", [[(4, 333)], [(2, 333), (3, 100)], [(4, 3000)]])
def test_few_rows_pages_of_no_keys(seqs, D, fmt):
    b = batch(seqs, 2, 4, D, 16, fmt, "bf16")
    last = (seqs[0][1] - 1) // 16  # that the tokens' own keys are in
    for page in (3, last):
        held = b.table[0, page]
        for bad in (-1, b.n_pages, -(1 << 31)):
            b.table[0, page] = bad
            b.check(b.run(), hidden={0: range(16 * page, min(16 * page + 16, seqs[0][1]))})
        b.table[0, page] = held
    b.table[0, :] = -7
    b.check(b.run(), hidden={0: range(seqs[0][1])})


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("D", [64, 128, 160])
@pytest.mark.parametrize("nq,nk", [(2, 70), (4, 66), (3, 400), (4, 3000)])
def test_few_rows_prefer_nothing_they_cannot_see(nq, nk, D, kind, fmt):
    """The last key: huge, a NaN block of its values and, in e4m3, NaN codes.  The
    last token's result is NaN, the others' as if the key were not there."""
    b = batch([(nq, nk)], 2, 4, D, 16, fmt, kind)
    last = b.slots[0][-1:]
    code = 0x7F if fmt == "fp8" else 0x77
    for i, scale in ((0, 240), (2, 255)):
        shape = b.pool.arrays[i].shape[-1]
        b.pool.put(i, last, np.full((1, 2, shape), code, np.uint8),
                   np.full((1, 2, D // 32), scale, np.uint8))
    b.pool.upload()
    y = host(b.run())
    assert np.isnan(y[1 + nq - 1]).all()
    # the tokens before the last as a sequence of their own, the key and its page gone
    b.seqs, b.most = [(nq - 1, nk - 1)], max(nq - 1, 1)
    b.starts = np.array([1, nq])
    b.slots[0] = b.slots[0][:-1]
    got = torch.from_numpy(y).clone()
    got[nq] = 31.0
    b.check(got)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("D,G,nq,nk", [(64, 2, 2, 70), (128, 4, 4, 400), (96, 2, 3, 64),
                                       (128, 4, 3, 2600), (256, 5, 3, 130)])
def test_few_rows_nan_reaches_those_that_see_it(D, G, nq, nk, kind, fmt):
    """NaN blocks of values in two of the chunk's own keys, each of one head and of
    32 dims; one of an older key's in a third place; a NaN key; a row of q that is
    not finite."""
    b = batch([(nq, nk)], 3, G, D, 16, fmt, kind, after=0, before=0)
    places = [(nk - 1, 0, 0), (nk - 2, 0, 1), (nk // 2, 1, D // 32 - 1)]  # key, head, block
    for key, h, block in places:
        s = b.slots[0][key]
        b.pool.arrays[3][s // 16, h, s % 16, block] = 255
    s = b.slots[0][nk - 2]
    b.pool.arrays[1][s // 16, 2, s % 16, D // 32 - 1] = 255
    b.pool.upload()
    b.q[0, 0, 3] = float("inf")
    b.held[0, 0, 3] = np.inf
    got = np.isnan(host(b.run()).reshape(nq, 3, G, D))
    sees = b.sees(0, True, 0)
    want = np.zeros_like(got)
    for key, h, block in places:
        want[:, h, :, 32 * block:32 * block + 32] |= sees[:, key][:, None, None]
    want[:, 2] |= sees[:, nk - 2][:, None, None]
    want[0, 0, 0] = True
    assert np.array_equal(got, want)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [64, 128])
def test_few_rows_powers_far_apart(D, kind, fmt):
    b = batch([(4, 100), (2, 300)], 2, 4, D, 16, fmt, kind)
    for i in (0, 1):
        n = len(b.slots[i])
        for a in (0, 2):
            x = b.g.standard_normal((n, 2, D)) * np.exp2(b.g.integers(-9, 10, (n, 2, D // 32))).repeat(32, -1)
            b.pool.put(a, b.slots[i], *mx.quantize(x, fmt))
    b.pool.upload()
    b.q, b.held = put(b.held * np.exp2(b.g.integers(-100, -6, (b.T, 8, 1))), kind)
    b.check(b.run())


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", list(TYPES))
def test_one_token_and_a_huge_key(kind, fmt):
    """The token's own key has the largest codes under 2^113 (e4m3: NaN codes): it
    takes all the weight where the score is positive, and e4m3 gives NaN."""
    b = Batch([(1, 45)], 2, 3, 64, 16, fmt, kind)
    code = 0x7F if fmt == "fp8" else 0x77
    shape = b.pool.arrays[0].shape[-1]
    b.pool.put(0, b.slots[0][-1:], np.full((1, 2, shape), code, np.uint8), np.full((1, 2, 2), 240, np.uint8))
    b.pool.upload()
    y = host(b.run())[1].reshape(2, 3, 64)
    if fmt == "fp8":
        assert np.isnan(y).all()
        return
    # The step's keys are taken with the huge key's power: the others beside it are
    # off by 2^-31 of it, 2^82, and their scores with it.  What is left of y where
    # the huge key has no weight is a mean of the values seen.
    score = b.held[1].reshape(2, 3, 64).sum(-1)
    v = b.pool.values(2, b.slots[0])
    most = np.abs(v).max(0)[:, None] * (1 + torch.finfo(TYPES[kind]).eps)
    assert (np.abs(y) <= np.broadcast_to(most, y.shape)).all()
    for h, r in np.argwhere(score > 0):  # one weight, exact but for y's rounding and two of fp32
        assert (np.abs(y[h, r] - v[-1, h]) <= (torch.finfo(TYPES[kind]).eps / 2 + 2.0 ** -22)
                * np.abs(v[-1, h])).all()
