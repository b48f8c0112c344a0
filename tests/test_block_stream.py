"""The stream that a call without one takes (CPU)."""
import torch

from routing_quant_expert_amd import binding


class Stream:
    cuda_stream = 4660


def test_current_stream_of_a_torch_without_the_raw_entry(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream())
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert binding._stream(None) == 4660


def test_current_stream_of_the_current_device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 100 + d, raising=False)
    assert binding._stream(None) == 103


def test_given_streams():
    assert binding._stream(Stream()) == 4660 and binding._stream(0) == 0 and binding._stream(7) == 7
