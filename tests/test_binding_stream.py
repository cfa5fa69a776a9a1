"""The stream that the binding takes when none is given, without torch's private names for it."""
import types

import pytest
import torch

from mixed_precision_quantized_mx_b200 import binding


@pytest.mark.parametrize("missing", ["_current_device", "_current_stream"])
def test_public_current_stream_where_a_private_name_is_missing(missing, monkeypatch):
    monkeypatch.setattr(binding, missing, None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=1234))
    assert binding._stream(None) == 1234
    assert binding._stream(77) == 77 and binding._stream(types.SimpleNamespace(cuda_stream=5)) == 5


def test_its_reason_where_there_is_no_stream(monkeypatch):
    def no_device():
        raise RuntimeError("no device")
    monkeypatch.setattr(binding, "_current_stream", None)
    monkeypatch.setattr(torch.cuda, "current_stream", no_device)
    with pytest.raises(RuntimeError, match="no device"):
        binding._stream(None)


@pytest.mark.gpu
def test_both_name_the_same_stream(monkeypatch):
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        fast = binding._stream(None)
        monkeypatch.setattr(binding, "_current_stream", None)
        assert binding._stream(None) == fast == side.cuda_stream
