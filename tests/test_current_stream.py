"""Calls without a stream: CUDA comes up with the first of them, or torch's own error says why it does not."""

import subprocess
import sys

import pytest
import torch

import bit_quantized_linear_hadamard_b200 as qs
from bit_quantized_linear_hadamard_b200 import binding


def test_without_cuda_torch_says_so(monkeypatch):
    def no_cuda(*_):
        raise AssertionError("Torch not compiled with CUDA enabled")

    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    for name in ("current_device", "current_stream"):
        monkeypatch.setattr(torch.cuda, name, no_cuda)
    with pytest.raises(AssertionError, match="not compiled with CUDA"):
        binding._s(None)


def test_without_the_short_way_to_the_stream(monkeypatch):
    class Stream:
        cuda_stream = 4711

    monkeypatch.setattr(binding, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: Stream if device == 3 else None)
    assert binding._s(None) == 4711


@pytest.mark.gpu
def test_the_first_call_of_a_process():
    code = ("import torch, bit_quantized_linear_hadamard_b200 as qs; assert not torch.cuda.is_initialized(); "
            "assert qs.qs_device_error() == 0 and torch.cuda.is_initialized(); "
            "s = torch.cuda.Stream(); torch.cuda.set_stream(s); from bit_quantized_linear_hadamard_b200 import binding; "
            "assert binding._s(None) == s.cuda_stream; print('ok')")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr
    assert binding._s(None) == torch.cuda.current_stream().cuda_stream
    assert qs.qs_device_error() == 0
