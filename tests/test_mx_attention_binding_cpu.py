"""What the attention operators' binding refuses before the C side is asked, with
stand-ins for GPU tensors (only their attributes are read)."""
import pytest
import torch

from q4_packed_weight_amd import binding


class Tensor:
    """A GPU tensor's attributes over a CPU one's."""

    def __init__(self, t, device=0):
        self.t, self.dtype, self.shape, self.is_cuda = t, t.dtype, t.shape, True
        self.device = torch.device("cuda", device)
        for name in ("numel", "is_contiguous", "data_ptr", "stride"):
            setattr(self, name, getattr(t, name))

    def get_device(self):
        return self.device.index


@pytest.fixture(autouse=True)
def device(monkeypatch):
    monkeypatch.setattr(binding, "_device", lambda: 0)


def rows(t, n, heads, head_dim):
    return binding._rows(Tensor(t), torch.float32, "x", n, heads, head_dim, 0)


def test_rows_of_both_shapes_and_strides():
    x = torch.zeros(4, 6, 32)
    assert rows(x, 4, 6, 32) == rows(x.view(4, 192), 4, 6, 32) == (x.data_ptr(), 192)
    assert rows(x[:, 2:4], 4, 2, 32) == (x[:, 2:4].data_ptr(), 192)
    assert rows(x.view(4, 192)[:, 64:128], 4, 2, 32) == (x[:, 2:4].data_ptr(), 192)
    assert rows(x[:1], 1, 6, 32)[1] == 192


@pytest.mark.parametrize("shape", [(4, 32, 6), (4, 2, 96), (4, 3, 2, 32), (4, 192, 1), (768,), (1, 4, 192),
                                   (24, 32)])
def test_rows_of_another_shape_are_refused(shape):
    """Contiguous ones too: [tokens][head_dim][heads] would be taken for heads."""
    with pytest.raises(ValueError):
        rows(torch.zeros(shape), 4, 6, 32)


def test_rows_that_do_not_lie_together_are_refused():
    x = torch.zeros(4, 6, 64)
    for t in (x[..., :32], x.transpose(1, 2)[:, :32], x[..., ::2], x.transpose(0, 1)[:4, :4].transpose(1, 2)):
        with pytest.raises(ValueError):
            rows(t, 4, t.shape[1], t.shape[2])


CALLS = {
    "mx_rotary": lambda f, i: binding.mx_rotary(f[0], i[0], f[1], 1.0, 2, 2, 32, 32, "half", f[0]),
    "mx_cache_write": lambda f, i: binding.mx_cache_write(f[0], f[0], i[0], 2, 2, 32, "fp8", *f[2:6], 4, 16),
    "mx_cache_read": lambda f, i: binding.mx_cache_read(i[0], 2, 2, 32, "fp8", *f[2:6], 4, 16, f[0], f[0]),
    "mx_attention": lambda f, i: binding.mx_attention(f[0], *i[1:4], 2, 2, 2, 32, 2, 2, 1, 1.0, True, 0, "fp8",
                                                      *f[2:6], 4, 16, f[0], f[6])}
USES = {"mx_rotary": ([0, 1], [0]), "mx_cache_write": ([0, 2, 3, 4, 5], [0]),
        "mx_cache_read": ([0, 2, 3, 4, 5], [0]), "mx_attention": ([0, 2, 3, 4, 5, 6], [1, 2, 3])}


@pytest.mark.parametrize("call,place", [(c, (k, n)) for c, u in USES.items() for k in (0, 1) for n in u[k]])
def test_tensors_of_another_device_are_refused(monkeypatch, call, place):
    """Each of them: nothing is launched."""
    def never(*a):
        raise AssertionError("launched")
    monkeypatch.setattr(binding, "_stream", lambda s: 0)
    lib = type("Lib", (), {call: never})
    monkeypatch.setattr(binding, "lib", lambda: lib)
    u8 = torch.zeros(4 * 2 * 16 * 32, dtype=torch.uint8)

    def tensors(other):
        f = [torch.zeros(2, 64), torch.zeros(16, dtype=torch.float64), u8, u8, u8, u8, u8]
        i = [torch.zeros(4, dtype=torch.int64)] + [torch.zeros(4, dtype=torch.int32)] * 3
        return [[Tensor(t, int(other == (k, n))) for n, t in enumerate(g)] for k, g in enumerate((f, i))]
    with pytest.raises(AssertionError, match="launched"):  # all on the current one
        CALLS[call](*tensors(None))
    with pytest.raises(ValueError, match="current device is another"):
        CALLS[call](*tensors(place))


def test_bands_and_yarn_have_their_own_defaults():
    """Bands lie between 1 turn over the trained positions and 4, YaRN's ramp between
    1 and 32; given ones are taken by both."""
    for scaling, high in (("bands", 4.0), ("yarn", 32.0)):
        f, _ = binding.mx_rotary_frequencies(128, 500000.0, scaling, 8.0)
        want, _ = binding.mx_rotary_frequencies(128, 500000.0, scaling, 8.0, 8192.0, 1.0, high)
        assert torch.equal(f, want)
        other, _ = binding.mx_rotary_frequencies(128, 500000.0, scaling, 8.0, high=9.0)
        assert not torch.equal(f, other)
    # turns over 8192 positions: 4 and more are kept, 1 and less are divided
    f, _ = binding.mx_rotary_frequencies(128, 500000.0, "bands", 8.0)
    plain, _ = binding.mx_rotary_frequencies(128, 500000.0)
    turns = 8192 * plain / 6.283185307179586
    assert torch.equal(f[turns >= 4], plain[turns >= 4])
    assert torch.allclose(f[turns <= 1], plain[turns <= 1] / 8, rtol=1e-15, atol=0)


@pytest.mark.parametrize("d", [514, 1 << 45, 1 << 62, -2, 0, 7])
def test_sizes_of_no_table_are_refused_without_one(d):
    with pytest.raises(binding.Q4KError) as e:
        binding.mx_rotary_frequencies(d)
    assert e.value.code == binding.Q4K_EINVAL_DIM
