"""The serving operators' binding on the host alone, without a GPU."""
import pytest
import torch

nv = pytest.importorskip("nvfp4_block_quantization_quantize_gb300")


class _Stream:
    def __init__(self, index):
        self.device = torch.device("cuda", index)


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """The work would run on the tensors' device's current stream, in no order with what the given one holds."""
    monkeypatch.setattr(torch.cuda, "Stream", _Stream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    dev = torch.device("cuda", 0)
    own = _Stream(0)
    assert nv._given_stream(own, dev) is own
    with pytest.raises(ValueError, match="stream"):
        nv._given_stream(_Stream(1), dev)
