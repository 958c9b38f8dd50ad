"""The attention operators without a GPU: the oracle against values worked by
hand, the frequency tables (host code), and every refusal of the C entry points
and of the binding (validation runs before any HIP call, so the fake pointers
are never read)."""
import ctypes
import math
import os

import numpy as np
import pytest

from oracle import mx


@pytest.fixture(scope="module")
def lib():
    from q4_packed_weight_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from q4_packed_weight_amd import build
        build.build()
    return binding.lib()


P = ctypes.c_void_p
PTR = [P(0x100000 * i) for i in range(1, 12)]
ODD = P(0x100004)
ODD2 = P(0x100002)
F32, BF16, FP4, FP8 = 0, 1, 4, 8


# ------------------------------------------------------------ the oracle

def test_rotary_turns_pairs():
    x = np.arange(1.0, 7.0).reshape(1, 1, 6)
    f = [math.pi / 2, math.pi]
    got = mx.rotary(x, [1], f, 1.0, 4, "half")[0, 0]
    assert np.allclose(got, [-3, -2, 1, -4, 5, 6])
    got = mx.rotary(x, [1], f, 2.0, 4, "interleaved")[0, 0]
    assert np.allclose(got, [-4, 2, -6, -8, 5, 6])


def test_attention_of_known_weights():
    k = np.array([[0.0], [math.log(3.0)], [50.0]])
    v = np.array([[1.0], [5.0], [1000.0]])
    sees = np.array([[1, 1, 0], [0, 0, 0], [1, 0, 0]], bool)
    y, mass, _, _ = mx.attention(np.ones((3, 1)), k, v, 1.0, sees)
    assert np.allclose(y[:, 0], [4.0, 0.0, 1.0]) and np.allclose(mass[:, 0], [4.0, 0.0, 1.0])


# ------------------------------------------------------------ frequencies

@pytest.mark.parametrize("d", [2, 4, 64, 96, 128, 512])
@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn", "bands"])
def test_frequencies_equal_the_definition(lib, scaling, d):
    from q4_packed_weight_amd import binding
    for base, factor, trained, low, high in ((10000.0, 4.0, 8192.0, 1.0, 32.0),
                                             (500000.0, 8.0, 4096.0, 1.0, 4.0),
                                             (10000.0, 1.0, 100.0, 2.0, 3.0)):
        f, a = binding.mx_rotary_frequencies(d, base, scaling, factor, trained, low, high)
        want, amp = mx.rotary_frequencies(d, base, scaling, factor, trained, low, high)
        assert f.shape == (d // 2,) and np.allclose(f.numpy(), want, rtol=1e-13, atol=0)
        assert abs(a - amp) < 1e-14


def test_frequencies_worked():
    from q4_packed_weight_amd import binding
    f, a = binding.mx_rotary_frequencies(4, 10000.0)
    assert np.allclose(f.numpy(), [1.0, 0.01]) and a == 1.0
    f, _ = binding.mx_rotary_frequencies(4, 10000.0, "linear", 4.0)
    assert np.allclose(f.numpy(), [0.25, 0.0025])
    f, _ = binding.mx_rotary_frequencies(4, 100.0, "ntk", 10.0)  # base 100 * 10^2
    assert np.allclose(f.numpy(), [1.0, 0.01])
    # 8192 positions: 1304 turns (kept) and 13.04: a share of (13.04 - 1) / 31
    f, _ = binding.mx_rotary_frequencies(4, 10000.0, "bands", 4.0, 8192.0, 1.0, 32.0)
    keep = (8192 * 0.01 / (2 * math.pi) - 1) / 31
    assert np.allclose(f.numpy(), [1.0, 0.01 * (keep + (1 - keep) / 4)])


def test_frequencies_refusals(lib):
    f, a = (ctypes.c_double * 256)(), ctypes.c_double()
    D = ctypes.c_double

    def call(d=64, base=1e4, scaling=0, factor=1.0, trained=8192.0, low=1.0, high=32.0, fp=f,
             ap=ctypes.byref(a)):
        return lib.mx_rotary_frequencies(d, D(base), scaling, D(factor), D(trained), D(low),
                                         D(high), fp, ap)
    assert call() == 0
    for d in (0, -2, 3, 514):
        assert call(d=d) == -1
    for s in (-1, 5):
        assert call(scaling=s) == -6
    for base in (1.0, 0.0, -3.0, math.inf, math.nan):
        assert call(base=base) == -1
    assert call(factor=0.5) == 0  # not read
    for s in (1, 2, 3, 4):
        for factor in (0.5, math.nan, math.inf):
            assert call(scaling=s, factor=factor) == -1
    for s in (3, 4):
        for k in ({"trained": 0.5}, {"trained": math.nan}, {"low": 0.0}, {"low": 32.0},
                  {"high": math.nan}, {"high": math.inf}):
            assert call(scaling=s, factor=2.0, **k) == -1
    assert call(fp=None) == -2 and call(ap=None) == -2


# ------------------------------------------------------------ refusals

def rotary(lib, x=PTR[0], xs=256, t=F32, pos=PTR[1], f=PTR[2], n=4, h=4, d=64, r=64, lay=0,
           y=PTR[3], ys=256):
    return lib.mx_rotary(x, xs, t, pos, f, ctypes.c_float(1), n, h, d, r, lay, y, ys, None)


def test_rotary_refusals(lib):
    for k in ({"n": 0}, {"n": -1}, {"n": 1 << 31}, {"h": 0}, {"h": 4097}, {"d": 0}, {"d": 60},
              {"d": 520, "r": 64}, {"r": 0}, {"r": 3}, {"r": 66}, {"r": -2}, {"xs": 255},
              {"ys": 255}, {"xs": 1 << 31}):
        assert rotary(lib, **k) == -1, k
    for k in ({"t": 3}, {"t": -1}, {"lay": 2}, {"lay": -1}):
        assert rotary(lib, **k) == -6, k
    for k in ({"x": None}, {"pos": None}, {"f": None}, {"y": None}):
        assert rotary(lib, **k) == -2, k
    for k in ({"x": ODD}, {"y": ODD}, {"pos": ODD}, {"f": ODD}, {"xs": 257}, {"ys": 258},
              {"t": BF16, "xs": 260}):
        assert rotary(lib, **k) == -3, k
    assert rotary(lib, x=None, t=9, d=3) == -1 and rotary(lib, x=None, t=9) == -6


def write(lib, k=PTR[0], ks=256, v=PTR[1], vs=256, t=F32, slots=PTR[2], n=4, h=4, d=64, f=FP8,
          pool=(PTR[3], PTR[4], PTR[5], PTR[6]), pages=8, size=16):
    return lib.mx_cache_write(k, ks, v, vs, t, slots, n, h, d, f, *pool, pages, size, None)


def read(lib, k=PTR[0], ks=256, v=PTR[1], vs=256, t=F32, slots=PTR[2], n=4, h=4, d=64, f=FP8,
         pool=(PTR[3], PTR[4], PTR[5], PTR[6]), pages=8, size=16):
    return lib.mx_cache_read(slots, n, h, d, f, *pool, pages, size, k, ks, v, vs, t, None)


@pytest.mark.parametrize("call", [write, read])
def test_cache_refusals(lib, call):
    for k in ({"n": 0}, {"n": -1}, {"n": 1 << 31}, {"h": 0}, {"h": 4097}, {"d": 0}, {"d": 48},
              {"d": 288}, {"ks": 255}, {"vs": 255}, {"pages": 0}, {"pages": 1 << 31},
              {"size": 0}, {"size": 65537}, {"pages": 1 << 20, "size": 1 << 11}):
        assert call(lib, **k) == -1, k
    for k in ({"t": 3}, {"f": 5}, {"f": 0}):
        assert call(lib, **k) == -6, k
    for name in ("k", "v", "slots"):
        assert call(lib, **{name: None}) == -2, name
    for i in range(4):
        pool = [PTR[3], PTR[4], PTR[5], PTR[6]]
        pool[i] = None
        assert call(lib, pool=pool) == -2, i
    for k in ({"k": ODD}, {"v": ODD}, {"slots": ODD}, {"ks": 258}, {"vs": 257},
              {"pool": (ODD, PTR[4], PTR[5], PTR[6])}, {"pool": (PTR[3], PTR[4], ODD, PTR[6])}):
        assert call(lib, **k) == -3, k


def attention(lib, q=PTR[0], qs=512, t=F32, starts=PTR[1], counts=PTR[2], table=PTR[3], n=4, h=8,
              hk=4, d=64, seqs=2, width=4, most=2, scale=0.125, causal=1, window=0, f=FP8,
              pool=(PTR[4], PTR[5], PTR[6], PTR[7]), pages=8, size=16, y=PTR[8], ys=512,
              ws=PTR[9], bytes=1 << 40):
    return lib.mx_attention(q, qs, t, starts, counts, table, n, h, hk, d, seqs, width, most,
                            ctypes.c_float(scale), causal, window, f, *pool, pages, size, y, ys,
                            ws, bytes, None)


BAD_SIZES = ({"n": 0}, {"n": 1 << 31}, {"h": 0}, {"h": 6}, {"h": 4100}, {"hk": 0}, {"hk": 3},
             {"d": 0}, {"d": 48}, {"d": 288}, {"seqs": 0}, {"seqs": -1}, {"width": 0},
             {"most": 0}, {"size": 0}, {"size": 65537}, {"width": 1 << 27, "size": 16},
             {"seqs": 1 << 23}, {"seqs": 1 << 12, "most": 1 << 16}, {"most": 1 << 30})


def test_attention_refusals(lib):
    for k in BAD_SIZES + ({"qs": 511}, {"ys": 511}, {"pages": 0}, {"pages": 1 << 31},
                          {"window": -1}, {"window": 4, "causal": 0},
                          {"scale": math.nan}, {"scale": math.inf}):
        assert attention(lib, **k) == -1, k
    for k in ({"t": 3}, {"f": 5}):
        assert attention(lib, **k) == -6, k
    for name in ("q", "starts", "counts", "table", "y"):
        assert attention(lib, **{name: None}) == -2, name
    for i in range(4):
        pool = [PTR[4], PTR[5], PTR[6], PTR[7]]
        pool[i] = None
        assert attention(lib, pool=pool) == -2, i
    for k in ({"q": ODD}, {"y": ODD}, {"starts": ODD2}, {"counts": ODD2}, {"table": ODD2},
              {"ws": P(0x100080)}, {"qs": 514}, {"ys": 513},
              {"pool": (ODD, PTR[5], PTR[6], PTR[7])}, {"pool": (PTR[4], PTR[5], ODD, PTR[7])}):
        assert attention(lib, **k) == -3, k
    assert attention(lib, q=None, t=9, d=3) == -1 and attention(lib, q=None, t=9) == -6


def test_attention_workspace(lib):
    def size(n=4, h=8, hk=4, d=64, seqs=2, width=4, most=2, size=16):
        return lib.mx_attention_workspace_size(n, h, hk, d, seqs, width, size, most)
    for k in BAD_SIZES:
        assert size(**k) == -1, k
    assert size() == 0  # few keys: one range
    big = size(n=2, most=1, width=4096)
    assert big > 0 and big % 256 == 0
    few = {"n": 2, "most": 1, "width": 4096}
    assert attention(lib, **few, bytes=big - 1) == -5
    assert b"mx_attention" in lib.q4k_strerror(-5)
    assert attention(lib, **few, ws=None) == -2


# ------------------------------------------------------------ the binding

def test_binding_refuses_what_it_marshals():
    import torch
    from q4_packed_weight_amd import binding
    x = torch.zeros(2, 64)
    u8 = torch.zeros(8192, dtype=torch.uint8)
    pos, f = torch.zeros(2, dtype=torch.int64), torch.zeros(16, dtype=torch.float64)
    with pytest.raises(ValueError):  # not a GPU tensor
        binding.mx_rotary(x, pos, f, 1.0, 2, 2, 32, 32, "half", x)
    with pytest.raises(ValueError):
        binding.mx_rotary(x, pos, f, 1.0, 2, 2, 32, 32, "quarter", x)
    with pytest.raises(TypeError):
        binding.mx_rotary(x.double(), pos, f, 1.0, 2, 2, 32, 32, "half", x)
    with pytest.raises(ValueError):
        binding.mx_rotary_frequencies(64, 1e4, "other")
    with pytest.raises(ValueError) as e:
        binding.mx_rotary_frequencies(63)
    assert e.value.code == binding.Q4K_EINVAL_DIM
    with pytest.raises(ValueError):
        binding.mx_cache_write(x, x, pos, 2, 2, 32, "fp6", u8, u8, u8, u8, 4, 16)
    with pytest.raises(ValueError):
        binding.mx_cache_read(pos, 2, 2, 32, "fp8", u8, u8, u8, u8, 4, 16, x, x)
    with pytest.raises(ValueError) as e:
        binding.mx_attention_workspace_size(4, 8, 3, 64, 2, 4, 16, 2)
    assert e.value.code == binding.Q4K_EINVAL_DIM
