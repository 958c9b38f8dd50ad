"""Rotary positions and cache rows beyond what one launch takes: 2^30 chunks of eight
values, 2^23 workgroups.  Bounds as in test_mx_attention_gpu.py."""
import numpy as np
import pytest
import torch

from oracle import mx
from q4_packed_weight_amd import binding
from gpu_util import DEV
from test_mx_attention_gpu import FILL, Pool, dev, host, rng, rotary_bound

pytestmark = pytest.mark.gpu

LAUNCH = 1 << 28  # tokens of one head of 32 dims
T = LAUNCH + 37
ROWS = np.array([0, 1, LAUNCH - 1, LAUNCH, LAUNCH + 20, T - 1])


def test_cache_write_beyond_one_launch():
    g = rng(41)
    rows = torch.from_numpy(g.standard_normal((len(ROWS), 32))).to(torch.bfloat16)
    x = torch.zeros(T, 32, dtype=torch.bfloat16, device=DEV)
    x[dev(ROWS)] = rows.to(DEV)
    pool = Pool(4, 1, 16, 32, "fp8")
    at = g.permutation(64)[:len(ROWS)]
    slots = torch.full((T,), -1, dtype=torch.int64, device=DEV)
    slots[dev(ROWS)] = dev(at)
    binding.mx_cache_write(x, x, slots, T, 1, 32, "fp8", *pool.t, 4, 16)
    codes, scales = mx.quantize(rows.double().numpy()[:, None], "fp8")
    for i in (0, 2):
        pool.put(i, at, codes, scales)
    for got, want in zip(pool.download(), pool.arrays):
        assert np.array_equal(got, want)


def test_cache_read_beyond_one_launch():
    g = rng(42)
    pool = Pool(4, 1, 16, 32, "fp8")
    for i in (1, 3):
        pool.arrays[i][:] = 124
    for i in (0, 2):
        pool.arrays[i] &= 0xF7  # no NaN codes
    pool.upload()
    at = g.permutation(64)[:len(ROWS)]
    slots = torch.full((T,), -1, dtype=torch.int64, device=DEV)
    slots[dev(ROWS)] = dev(at)
    k, v = (torch.full((T, 32), FILL, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    binding.mx_cache_read(slots, T, 1, 32, "fp8", *pool.t, 4, 16, k, v)
    for got, i in ((k, 0), (v, 2)):
        assert np.array_equal(host(got[dev(ROWS)]), pool.values(i, at)[:, 0])
        got[dev(ROWS)] = 0
        for part in got.split(1 << 26):
            assert not part.any()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("R", [512, 510])
def test_rotary_beyond_one_launch(R, layout):
    """One token a workgroup, whole chunks and single pairs, in place."""
    launch = 1 << 23
    n = launch + 5
    rows = np.array([0, launch - 1, launch, n - 1])
    g = rng(43)
    x = torch.zeros(n, 512, dtype=torch.bfloat16, device=DEV)
    held = torch.from_numpy(g.standard_normal((4, 512))).to(torch.bfloat16)
    x[dev(rows)] = held.to(DEV)
    pos = torch.arange(n, device=DEV) * 3
    f, _ = binding.mx_rotary_frequencies(R)
    binding.mx_rotary(x, pos, f.to(DEV), 1.5, n, 1, 512, R, layout, x)
    held = held.double().numpy()[:, None]
    want = mx.rotary(held, rows * 3, f.numpy(), 1.5, R, layout)
    got = host(x[dev(rows)])[:, None]
    assert (np.abs(got - want) <= rotary_bound(want, held, 1.5, R, layout, "bf16")).all()
    x[dev(rows)] = 0
    for part in x.split(1 << 21):
        assert not part.any()
