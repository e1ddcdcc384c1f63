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
