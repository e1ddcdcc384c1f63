"""The serving operators' binding on the host alone, without a GPU."""
import sys
import types

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


def without_short_path(monkeypatch, module):
    """The package as a new process finds it, with `module` in the short path's place (None: its import fails)."""
    nv.build()
    monkeypatch.setattr(nv, "_lib", None)
    monkeypatch.setattr(nv, "_call", None)
    monkeypatch.setitem(sys.modules, nv.__name__ + "._nvfp4_call", module)
    if hasattr(nv, "_nvfp4_call"):
        monkeypatch.delattr(nv, "_nvfp4_call")


def still_works():
    assert nv.load_library().nvfp4_abi_version() > 0
    x, u = torch.zeros(2, 64), torch.zeros(2, 32, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):         # the Python checks take the calls
        nv.nvfp4_rmsnorm(x)
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_mv(x, u, u)
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_grouped_mm(u, u, torch.zeros(2, dtype=torch.int64), u[None], u[None])


def test_the_library_loads_without_the_short_path(monkeypatch):
    """Quantization does not need it: a file that does not load (another torch) costs the serving calls some
    microseconds, and nobody the library."""
    without_short_path(monkeypatch, None)
    with pytest.warns(RuntimeWarning, match="short call path"):
        nv.load_library()
    still_works()


def test_a_short_path_for_another_torch_is_not_used(monkeypatch):
    """It reads tensors by the layouts it was compiled with."""
    def bind(*args):
        raise AssertionError("bound")

    old = types.ModuleType("_nvfp4_call")
    old.abi, old.bind = "torch 1.0, cpython-38", bind
    without_short_path(monkeypatch, old)
    with pytest.warns(RuntimeWarning, match="built for torch 1.0"):
        nv.load_library()
    still_works()


def test_a_build_for_another_torch_or_interpreter_is_stale(monkeypatch):
    nv.build()
    mod = sys.modules[nv.__name__ + ".build"]
    assert not mod.is_stale()
    monkeypatch.setattr(torch, "__version__", "1.0")
    assert mod.is_stale()
    monkeypatch.undo()
    monkeypatch.setattr(mod.sysconfig, "get_config_var", lambda n: "cpython-38")
    assert mod.is_stale()
