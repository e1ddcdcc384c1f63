"""What a call of a serving operator takes and how it fails: the binding's short
path (csrc/nvfp4_call.cpp) against the Python one."""
import numpy as np
import pytest
import torch

import nvfp4_workloads as W
from parity_helpers import to_dev

pytestmark = pytest.mark.gpu

nv = pytest.importorskip("nvfp4_block_quantization_quantize_gb300")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    nv.build()
    nv.load_library()


@pytest.mark.parametrize("want", [1, np.bool_(True), "yes", 0, None, np.bool_(False)])
def test_want_out_is_a_truth_value(want):
    """Whatever its type, and whichever path the call takes."""
    x = to_dev(W.matrix((3, 64), seed=1, dtype="bf16"))
    short = nv.nvfp4_rmsnorm(x, want_out=want)
    long = nv.nvfp4_rmsnorm(x, want_out=want, stream=torch.cuda.current_stream())
    assert set(short) == set(long) == {"codes", "scales"} | ({"out"} if want else set())


def test_a_failed_allocation_is_an_out_of_memory_error():
    """As the caching allocator raises it, so that a caller may free memory and try again.  (The limit is the
    process's own: the output is 256 MB, of a card that has hundreds of times as much.)"""
    x = torch.zeros((16, 16), device="cuda")
    codes = torch.zeros((1 << 22, 8), device="cuda", dtype=torch.uint8)
    scales = torch.zeros((1 << 22, 1), device="cuda", dtype=torch.uint8)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (64 << 20)) / total)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            nv.nvfp4_mv(x, codes, scales, out_dtype="f32")
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    y = nv.nvfp4_mv(x, codes, scales, out_dtype="f32")
    assert bool((y == 0).all())
