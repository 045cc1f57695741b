"""The binding's current stream (CPU only: torch's functions are stood in for)."""
from types import SimpleNamespace

import pytest
import torch

from long_context_serving_gb300 import bsattn as B


@pytest.mark.parametrize("gone", [(), ("_cuda_getCurrentRawStream",), ("_cuda_getDevice",)])
def test_current_stream_without_torch_internals(monkeypatch, gone):
    """The raw handle comes from torch's internals, or, on a torch without them, from its Stream."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0x100 + d, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: SimpleNamespace(cuda_stream=0x200))
    for name in gone:
        monkeypatch.delattr(torch._C, name)
    monkeypatch.setattr(B, "_current", B._current_stream())
    assert B._stream(None) == (0x200 if gone else 0x103)
    assert B._stream(7) == 7 and B._stream(SimpleNamespace(cuda_stream=9)) == 9
