"""The stream that a call without one goes to: the current stream's handle, by torch's short way
where this torch has it and by the Stream object where it has not."""
import importlib.util
import types

import pytest
import torch

from paged_kv_cache_90_gb300 import binding


def _fresh(monkeypatch):
    spec = importlib.util.spec_from_file_location("paged_kv_cache_90_gb300.binding_copy", binding.__file__)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m._have_cuda = True
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=42 + (device or 0)))
    return m


def test_current_stream_without_the_short_way(monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert _fresh(monkeypatch)._stream(None).value == 45


def test_current_stream_by_the_short_way(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 100 + device, raising=False)
    m = _fresh(monkeypatch)
    assert m._stream(None).value == 103
    assert m._stream(7).value == 7


@pytest.mark.gpu
def test_current_stream_is_the_one_that_torch_reports():
    assert (binding._stream(None).value or 0) == torch.cuda.current_stream().cuda_stream
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        assert binding._stream(None).value == s.cuda_stream
    assert binding._stream(s).value == s.cuda_stream
