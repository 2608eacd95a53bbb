"""How the serving binding finds the current stream, on the CPU: torch's quick
entry point where it is there, the public one where it is not."""
import importlib.util

import torch

from post_weight_quantization_row_amd import serve


def load_again():
    spec = importlib.util.spec_from_file_location(serve.__package__ + ".serve_again", serve.__file__)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


class _Stream:
    cuda_stream = 1234


def launches(module, monkeypatch, current, device):
    """(handle, the device that was current) of a call on the current stream."""
    seen = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current)

    class guard:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            seen.append(self.device)

        def __exit__(self, *exc):
            pass

    monkeypatch.setattr(torch.cuda, "device", guard)
    module._call(torch.device("cuda", device), None, lambda *a: seen.append(a) or 0, "x")
    return seen


def test_without_the_quick_entry_point(monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    asked = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda i: asked.append(i) or _Stream)
    again = load_again()
    assert launches(again, monkeypatch, 0, 0) == [("x", 1234)]
    assert launches(again, monkeypatch, 0, 1) == [torch.device("cuda", 1), ("x", 1234)]
    assert asked == [0, 1]


def test_with_it(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 77 + i, raising=False)
    assert launches(load_again(), monkeypatch, 1, 1) == [("x", 78)]
