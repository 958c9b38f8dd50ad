"""The binding where torch is built without a GPU: importing it needs none, and
the current stream is then torch's public one (which says what is missing)."""
import importlib.util
import types

import pytest
import torch

from q4_packed_weight_amd import binding

PRIVATE = ("_cuda_getCurrentRawStream", "_cuda_getDevice")


@pytest.mark.parametrize("missing", [PRIVATE[:1], PRIVATE[1:], PRIVATE])
def test_import_without_torchs_gpu_names(monkeypatch, missing):
    for name in missing:
        monkeypatch.delattr(torch._C, name)
    spec = importlib.util.spec_from_file_location("binding_without_gpu", binding.__file__)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=77))
    assert m._stream(None) == 77
    assert m._stream(types.SimpleNamespace(cuda_stream=5)) == 5
