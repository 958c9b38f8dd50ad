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
    monkeypatch.setattr(binding, "_current_device", lambda: 0)


def rows(t, n, heads, head_dim):
    return binding._rows(Tensor(t), torch.float32, "x", n, heads, head_dim)


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
