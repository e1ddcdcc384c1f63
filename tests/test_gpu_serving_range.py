"""What nvfp4_mv keeps of activations that lie far below others of their token.

x enters the product in f16 after a power-of-two scaling to the largest magnitude
of a part of its columns: a bf16 or MXFP8 element is off by at most 2^-39 of that
magnitude (half an f16 step of 2^-24 on values scaled to [2^14, 2^15)), an fp32 one,
held as two f16, by 2^-23 of itself or 2^-50 of that magnitude (half a step of the
second, which stands for 2^-11 of the first's).  Weights that are zero where x is large let the
small elements alone reach the output, so nothing hides what was lost.
"""
import numpy as np
import pytest
import torch

import oracle
from parity_helpers import to_dev, to_np

pytestmark = pytest.mark.gpu

nv = pytest.importorskip("nvfp4_block_quantization_quantize_gb300")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    nv.build()
    nv.load_library()


def weight(rng, N, K, zero_columns):
    """Random codes, zero at the columns given; scales 1/2, 1 and 2; and their float64 values."""
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    low, high = codes & 15, codes >> 4
    low[:, zero_columns[0::2]] = 0
    high[:, zero_columns[1::2]] = 0
    codes = (low | high << 4).astype(np.uint8)
    scales = (0x38 + 8 * rng.integers(-1, 2, (N, K // 16))).astype(np.uint8)
    return codes, scales, oracle.dequantize(codes, scales, N, K, out_dtype=oracle.F32).astype(np.float64)


def e4m3(values):
    return torch.from_numpy(np.asarray(values, np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


@pytest.mark.parametrize("gap", [0, 10, 22, 24, 25, 26, 31, 36, 40, 46, 60])
@pytest.mark.parametrize("top_code", [2.0 ** -9, 7 * 2.0 ** -9, 2.0 ** -6, 1.0, 448.0])
@pytest.mark.parametrize("M,K", [(1, 512), (9, 2064)])
def test_mv_mxfp8_keeps_what_is_near_the_largest_value(gap, top_code, M, K):
    """Groups whose scales are `gap` powers of two below the top one's, with codes of all sizes; the top group holds
    one value alone, top_code, where the weights are zero."""
    rng = np.random.default_rng(gap + K)
    N = 40
    codes, scales, w = weight(rng, N, K, np.array([0]))
    groups = -(-K // 32)
    x = rng.choice(np.array([2.0 ** -9, 3 * 2.0 ** -9, 0.5, 1.75, 15.0, 448.0, 0.0], np.float32), (M, K))
    x *= rng.choice(np.float32([-1, 1]), (M, K))
    x[:, :32] = 0.0
    x[:, 0] = top_code
    b = np.full((M, groups), 150 - gap, np.uint8)
    b[:, 0] = 150
    xv = x.astype(np.float64) * np.repeat(2.0 ** (b.astype(np.float64) - 127), 32, axis=1)[:, :K]
    y = nv.nvfp4_mv(to_dev(e4m3(x)), to_dev(codes), to_dev(scales), x_scales=to_dev(b), out_dtype="f32")
    top = np.abs(xv).max(axis=1, keepdims=True)
    # at most 2^-39 of the token's largest value an element (a part's is no larger), and the fp32 sums
    bound = (np.full_like(xv, 2.0 ** -39) * top) @ np.abs(w).T + (np.abs(xv) @ np.abs(w).T) * (17 * 2.0 ** -22)
    assert (np.abs(to_np(y).astype(np.float64) - xv @ w.T) <= bound).all()


def test_mv_mxfp8_far_ends_of_the_scales():
    """The smallest element of the smallest scale alone, the largest of the largest, and both in two tokens."""
    rng = np.random.default_rng(3)
    N, K = 33, 256
    codes, scales, w = weight(rng, N, K, np.array([], int))
    x, b = np.zeros((4, K), np.float32), np.full((4, K // 32), 127, np.uint8)
    x[0, 5], b[0, 0] = 2.0 ** -9, 0
    x[1, 70], b[1, 2] = 448.0, 240                        # 448 * 2^113 * 12 is below fp32's end
    x[2, 5], b[2, 0] = 2.0 ** -9, 250
    x[2, 70], b[2, 2] = 448.0, 232
    x[3, 200] = -0.875
    xv = x.astype(np.float64) * np.repeat(2.0 ** (b.astype(np.float64) - 127), 32, axis=1)
    y = to_np(nv.nvfp4_mv(to_dev(e4m3(x)), to_dev(codes), to_dev(scales), x_scales=to_dev(b), out_dtype="f32"))
    want = (xv @ w.T).astype(np.float32)                  # one or two products: exact in fp32
    assert np.array_equal(y, want)


@pytest.mark.parametrize("gap", [0, 12, 15, 18, 20, 25, 27, 30, 35, 40, 60])
@pytest.mark.parametrize("M,K", [(1, 512), (9, 2064)])
@pytest.mark.parametrize("x_type", ["f32", "bf16"])
def test_mv_keeps_what_is_near_the_largest_value(gap, M, K, x_type):
    """One value 2^gap times the others' size, where the weights are zero."""
    rng = np.random.default_rng(gap + K)
    N = 40
    codes, scales, w = weight(rng, N, K, np.array([0]))
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[:, 0] = 1.25 * 2.0 ** gap
    xd = torch.from_numpy(x).cuda().to(torch.float32 if x_type == "f32" else torch.bfloat16)
    xv = xd.double().cpu().numpy()
    y = nv.nvfp4_mv(xd, to_dev(codes), to_dev(scales), out_dtype="f32")
    top = np.abs(xv).max(axis=1, keepdims=True)
    off = np.maximum(np.abs(xv) * 2.0 ** -23, top * 2.0 ** -50) if x_type == "f32" else np.full_like(xv, 2.0 ** -39) * top
    bound = off @ np.abs(w).T + (np.abs(xv[:, 1:]) @ np.abs(w[:, 1:]).T) * (17 * 2.0 ** -22)
    assert (np.abs(to_np(y).astype(np.float64) - xv @ w.T) <= bound).all()
