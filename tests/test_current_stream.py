"""The stream that calls without one run on (CPU only, torch's answers stood in for)."""
import types

import pytest

torch = pytest.importorskip("torch")
from token_dispatch_grouped_amd import _lib  # noqa: E402


@pytest.fixture
def gpu(monkeypatch):
    monkeypatch.setattr(_lib, "_stream_query", None)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "init", lambda: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=77))


@pytest.mark.parametrize("missing", ["_cuda_getCurrentRawStream", "_cuda_getDevice"])
def test_a_torch_without_the_short_way(gpu, monkeypatch, missing):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 55, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.delattr(torch._C, missing)
    assert [_lib.current_stream() for _ in range(2)] == [77, 77]


def test_the_short_way_asks_for_the_current_device_each_time(gpu, monkeypatch):
    now = [0]
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 100 + device, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    assert _lib.current_stream() == 100
    now[0] = 3
    assert _lib.current_stream() == 103


def test_no_gpu_is_no_stream(monkeypatch):
    monkeypatch.setattr(_lib, "_stream_query", None)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: False)
    assert _lib.current_stream() is None
