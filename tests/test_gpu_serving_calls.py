"""What a call of a serving operator takes and how it fails: the binding's short
path (csrc/nvfp4_call.cpp) against the Python one, and the layers on batches of
no rows."""
import ctypes
import shutil
import subprocess
import threading

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


STUB = r"""
#include <stdint.h>
#include <time.h>
static volatile int flag = 0;
void set_flag(void) { flag = 1; }
/* stands for nvfp4_mv's launch: returns NVFP4_OK when another thread has set the flag, NVFP4_ECUDA after 5 s without */
int slow(void) {
    struct timespec t = {0, 1000000};
    for (int i = 0; i < 5000; ++i) {
        if (flag) return 0;
        nanosleep(&t, 0);
    }
    return 2;
}
"""


def test_other_threads_run_while_a_call_waits(tmp_path):
    """A launch may block (a full queue) until something that another Python thread does: the interpreter's lock is
    not held meanwhile, as ctypes does not hold it.  (The library's function is replaced by one that waits.)"""
    cc = shutil.which("gcc") or shutil.which("cc")
    src, lib = tmp_path / "stub.c", tmp_path / "stub.so"
    src.write_text(STUB)
    subprocess.run([cc, "-shared", "-fPIC", "-o", str(lib), str(src)], check=True)
    stub, real = ctypes.CDLL(str(lib)), nv.load_library()
    addr = lambda f: ctypes.cast(f, ctypes.c_void_p).value                       # noqa: E731
    own = [addr(f) for f in (real.nvfp4_rmsnorm, real.nvfp4_mv, real.nvfp4_grouped_mm, real.nvfp4_grouped_mm_workspace)]
    q = nv.nvfp4_quantize(to_dev(W.matrix((32, 64), seed=1, dtype="bf16")))
    x = to_dev(W.matrix((2, 64), seed=2, dtype="bf16"))
    nv._call.bind(own[0], addr(stub.slow), own[2], own[3])
    try:
        t = threading.Timer(0.05, stub.set_flag)
        t.start()
        y = nv._call.mv(x, q["codes"], q["scales"], None, None, 448.0, "bf16", None)
        t.join()
    finally:
        nv._call.bind(*own)
    assert y is not None                                  # None: the flag was not set within the wait


def test_experts_of_an_empty_batch():
    from nvfp4_block_quantization_quantize_gb300.serving import FP4Experts, FP4Projection
    r = lambda *s: torch.randn(*s, device="cuda").to(torch.bfloat16)             # noqa: E731
    layer = FP4Experts(r(128), r(4, 128), r(4, 128, 128), r(4, 128, 64), top_k=2)
    out, hidden = layer(r(0, 128), r(0, 128))
    assert out.shape == hidden.shape == (0, 128) and out.dtype == hidden.dtype == torch.bfloat16
    y, hidden = FP4Projection(r(96, 128), r(128))(r(0, 128), r(0, 128))
    assert y.shape == (0, 96) and hidden.shape == (0, 128)


@pytest.mark.parametrize("activations", ["mxfp8", "nvfp4"])
def test_projection_precision_does_not_go_by_the_batch(activations):
    """A token's product is of the same quantized activations whatever it comes with: alone and in batches it is the
    same sum of exact products, in orders that may differ by an fp32 step each (2^-17 of the magnitudes on both
    sides, as test_gpu_serving_layers.py has it)."""
    from nvfp4_block_quantization_quantize_gb300.serving import FP4Projection
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen).to(torch.bfloat16)      # noqa: E731
    N, K, M = 200, 512, 70
    w, nw, x, h = r(N, K), r(K), r(M, K), r(M, K)
    layer = FP4Projection(w, nw, activations=activations)
    if activations == "mxfp8":
        n = nv.nvfp4_rmsnorm(x, nw, hidden=h)
        mag = n["codes"].view(torch.float8_e4m3fn).double().abs() * torch.pow(2.0, n["scales"].double() - 127).repeat_interleave(32, 1)
    else:
        n = nv.nvfp4_rmsnorm(x, nw, hidden=h, format="nvfp4", gamax_mode="row")
        mag = nv.nvfp4_dequantize(n["codes"], n["scales"], M, K, gamax=n["gamax"], gamax_mode="row_given",
                                  out_dtype="f32").double().abs()
    q = nv.nvfp4_quantize(w, gamax_mode="tensor")
    wv = nv.nvfp4_dequantize(q["codes"], q["scales"], N, K, gamax=q["gamax"], gamax_mode="tensor_given", out_dtype="f32")
    bound = 2 * (mag @ wv.double().abs().t()) * 2.0 ** -17
    whole, hidden = layer(x, h, out_dtype="f32")
    assert whole.shape == (M, N) and torch.equal(hidden, (x.float() + h.float()).to(x.dtype))
    for a, b in ((0, 1), (3, 19), (16, 33), (69, 70)):
        part, _ = layer(x[a:b], h[a:b], out_dtype="f32")
        assert bool(((part.double() - whole[a:b].double()).abs() <= bound[a:b]).all())
    with pytest.raises(ValueError, match="activations"):
        FP4Projection(w, nw, activations="fp8")
