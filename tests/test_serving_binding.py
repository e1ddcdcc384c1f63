"""The serving operators' binding on the host alone, without a GPU."""
import sys

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


def test_the_library_is_published_last(monkeypatch):
    """Other threads read the library without the lock and then use the short path: at no step of loading is the
    first there without the second."""
    nv.build()
    nv.load_library()
    monkeypatch.setattr(nv, "_lib", None)
    monkeypatch.setattr(nv, "_call", None)
    seen = []

    def trace(frame, event, arg):
        if frame.f_code is not nv.load_library.__code__:
            return None
        if not frame.f_trace_opcodes:
            frame.f_trace_opcodes = True
            sys.settrace(trace)                           # some interpreters look at the flag here alone
        seen.append((nv._lib is None, nv._call is None))
        return trace

    old = sys.gettrace()
    sys.settrace(trace)
    try:
        nv.load_library()
    finally:
        sys.settrace(old)
    assert len(seen) > 100 and (False, True) not in seen
    assert nv._lib is not None and nv._call is not None
