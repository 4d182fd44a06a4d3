"""The binding's default stream is torch's current one, with and without the
torch function that gives its handle directly.  CPU only, with stand-ins."""
from types import SimpleNamespace

import torch

import mixture_experts_layer_gemv_amd as M


def test_without_the_raw_stream_function(monkeypatch):
    monkeypatch.setattr(M, "_current_stream", None, raising=False)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    handles = iter([77, 78])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: SimpleNamespace(cuda_stream=next(handles)))
    assert M._s(None) == 77 and M._s(None) == 78  # asked at each call


def test_with_the_raw_stream_function(monkeypatch):
    monkeypatch.setattr(M, "_current_stream", None, raising=False)
    devices = iter([1, 3])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 100 + d, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: next(devices))
    assert M._s(None) == 101 and M._s(None) == 103  # of the device that is current at each call


def test_given_streams():
    assert M._s(5) == 5 and M._s(SimpleNamespace(cuda_stream=9)) == 9
