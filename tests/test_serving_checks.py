"""Refusals of the serving operators, checked without a GPU: the C ABI's
argument checks run on the host before any CUDA call, the binding's before the
library is called."""
import ctypes

import pytest
import torch

nv = pytest.importorskip("nvfp4_block_quantization_quantize_gb300")

A16 = ctypes.c_void_p(0x10000)          # never used as an address: every call below is refused or empty
A8 = ctypes.c_void_p(0x10008)
A4 = ctypes.c_void_p(0x10004)
ODD = ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def lib():
    nv.build()
    return nv.load_library()


def norm(lib, x=A16, hidden=None, M=4, K=64, dtype=1, weight=None, wdt=1, eps=1e-6, hidden_out=None, out=None,
         fmt=1, gm=0, gamax=None, bound=448.0, codes=A16, scales=A16):
    return lib.nvfp4_rmsnorm(x, hidden, M, K, dtype, weight, wdt, eps, hidden_out, out, fmt, gm, gamax, bound, codes,
                             scales, None)


NORM_BAD = {
    "K not a multiple of 16": dict(K=72),
    "negative M": dict(M=-1),
    "bad dtype": dict(dtype=2),
    "bad weight dtype": dict(weight=A16, wdt=5),
    "negative eps": dict(eps=-1.0),
    "eps NaN": dict(eps=float("nan")),
    "eps infinite": dict(eps=float("inf")),
    "bad format": dict(fmt=2),
    "computed tensor amax": dict(fmt=0, gm=1, gamax=A16),
    "gamax with mxfp8": dict(gm=3, gamax=A16),
    "gamax NULL": dict(fmt=0, gm=2),
    "gamax misaligned": dict(fmt=0, gm=2, gamax=ODD),
    "bad gamax mode": dict(fmt=0, gm=7, gamax=A16),
    "bound zero": dict(bound=0.0),
    "bound NaN": dict(bound=float("nan")),
    "codes without scales": dict(scales=None),
    "no output": dict(codes=None, scales=None),
    "gamax without codes": dict(codes=None, scales=None, out=A16, fmt=0, gm=2, gamax=A16),
    "hidden without hidden_out": dict(hidden=A16),
    "hidden_out without hidden": dict(hidden_out=A16),
    "x NULL": dict(x=None),
    "hidden_out is x": dict(hidden=ctypes.c_void_p(0x20000), hidden_out=A16),
    "out is x": dict(out=A16),
    "x misaligned": dict(x=A8),
    "weight misaligned": dict(weight=A8),
    "codes misaligned": dict(codes=A8),
}


@pytest.mark.parametrize("case", sorted(NORM_BAD))
def test_norm_rejects(lib, case):
    assert norm(lib, **NORM_BAD[case]) == 1
    assert lib.nvfp4_last_error() != b""


def mv(lib, x=A16, xs=None, xt=1, codes=A16, scales=A16, M=4, N=32, K=64, gm=0, gamax=None, bound=448.0, out=A16,
       odt=1):
    return lib.nvfp4_mv(x, xs, xt, codes, scales, M, N, K, gm, gamax, bound, out, odt, None)


MV_BAD = {
    "17 rows": dict(M=17),
    "negative N": dict(N=-1),
    "K not a multiple of 16": dict(K=72),
    "N of 2^30": dict(N=1 << 30),
    "bad x type": dict(xt=3),
    "mxfp8 without scales": dict(xt=2),
    "scales without mxfp8": dict(xs=A16),
    "computed amax": dict(gm=1, gamax=A16),
    "gamax NULL": dict(gm=3),
    "gamax misaligned": dict(gm=4, gamax=ODD),
    "bound above 448": dict(bound=500.0),
    "bad out dtype": dict(odt=2),
    "x NULL": dict(x=None),
    "codes NULL": dict(codes=None),
    "scales misaligned": dict(scales=A8),
    "out NULL": dict(out=None),
}


@pytest.mark.parametrize("case", sorted(MV_BAD))
def test_mv_rejects(lib, case):
    assert mv(lib, **MV_BAD[case]) == 1
    assert lib.nvfp4_last_error() != b""


def grouped(lib, ca=A16, sa=A16, off=A16, cb=A16, sb=A16, E=4, T=8, N=32, K=64, gm=0, ga=None, gb=None, bound=448.0,
            out=A16, odt=1, ws=None, ws_bytes=0):
    return lib.nvfp4_grouped_mm(ca, sa, off, cb, sb, E, T, N, K, gm, ga, gb, bound, out, odt, ws, ws_bytes, None)


GROUPED_BAD = {
    "K not a multiple of 64": dict(K=96),
    "negative E": dict(E=-1),
    "E * N of 2^30": dict(E=1 << 16, N=1 << 14),
    "T of 2^30": dict(T=1 << 30),
    "computed amax": dict(gm=2, ga=A16),
    "gamax_a NULL": dict(gm=3),
    "gamax_b misaligned": dict(gb=ODD),
    "bound zero": dict(bound=0.0),
    "bad out dtype": dict(odt=9),
    "codes_a NULL": dict(ca=None),
    "scales_b NULL": dict(sb=None),
    "offsets NULL": dict(off=None),
    "offsets misaligned": dict(off=A4),
    "codes_b misaligned": dict(cb=A8),
    "out NULL": dict(out=None),
    "workspace too small": dict(E=8, T=8192, N=14336, K=4096, ws=A16, ws_bytes=64),
    "workspace NULL": dict(E=8, T=8192, N=14336, K=4096, ws_bytes=1 << 40),
    "workspace misaligned": dict(E=8, T=8192, N=14336, K=4096, ws=A8, ws_bytes=1 << 40),
}


@pytest.mark.parametrize("case", sorted(GROUPED_BAD))
def test_grouped_rejects(lib, case):
    assert grouped(lib, **GROUPED_BAD[case]) == 1
    assert lib.nvfp4_last_error() != b""


def test_workspace_is_asked_for_by_the_sizes(lib):
    assert lib.nvfp4_grouped_mm_workspace(64, 64, 2048, 4096) == 0
    assert lib.nvfp4_grouped_mm_workspace(8, 8192, 14336, 4096) == (8192 // 192 + 8) * 64 * 1024
    for bad in ((0, 1, 1, 64), (1, -1, 1, 64), (1 << 31, 1, 1, 64)):
        assert lib.nvfp4_grouped_mm_workspace(*bad) == 0


def test_empty_calls_are_valid(lib):
    assert norm(lib, M=0, x=None, codes=None, scales=None) == 0
    assert mv(lib, M=0, x=None, out=None) == 0
    assert mv(lib, N=0, codes=None, scales=None, out=None) == 0
    assert grouped(lib, T=0, ca=None, sa=None, out=None) == 0
    assert grouped(lib, E=0, off=None, cb=None, sb=None) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 64)
    u = torch.zeros(2, 32, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_rmsnorm(x)
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_mv(x, u, u)
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_grouped_mm(u, u, torch.zeros(2, dtype=torch.int64), u[None], u[None])
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_grouped_scales_to_mma(u[None])
