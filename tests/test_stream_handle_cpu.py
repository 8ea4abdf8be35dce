"""The stream handle that every entry point passes on: the given stream's, else
the current stream's, with or without torch's short cut to it."""
from types import SimpleNamespace

import pytest

import sigmoid_top_routing_router_amd as M


def fake_torch(**short_cut):
    current = SimpleNamespace(cuda_stream=0x5000)
    return SimpleNamespace(_C=SimpleNamespace(**short_cut),
                           cuda=SimpleNamespace(current_device=lambda: 3,
                                                current_stream=lambda: current))


@pytest.mark.parametrize("short_cut", [{}, {"_cuda_getCurrentRawStream": lambda d: 0x4FFD + d}])
def test_current_stream(monkeypatch, short_cut):
    monkeypatch.setattr(M, "_torch_module", fake_torch(**short_cut))
    assert M._stream(None).value == 0x5000
    assert M._stream(SimpleNamespace(cuda_stream=0x6000)).value == 0x6000
