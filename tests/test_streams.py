"""The stream that a call without one goes to."""
import types

import pytest
import torch

from lfsr_seeded_moe_b200 import nslm


def test_the_current_stream_of_a_torch_without_raw_handles(monkeypatch):
    # the raw handle is not part of torch's public interface
    monkeypatch.setattr(nslm, "_current_stream", None, raising=False)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=4711))
    assert nslm._s(None) == 4711
    assert nslm._s(12) == 12
    assert nslm._s(types.SimpleNamespace(cuda_stream=13)) == 13


@pytest.mark.gpu
def test_the_current_stream_is_looked_up_at_each_call():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    assert nslm._s(None) == torch.cuda.current_stream().cuda_stream
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert nslm._s(None) == side.cuda_stream
    assert nslm._s(None) == torch.cuda.current_stream().cuda_stream
