"""An output of a serving operator that shares a byte with an input or another
output is refused on the host, before any CUDA call (the hidden state alone may
be updated in place).  The addresses below are never used: every call is refused."""
import ctypes

import pytest
import torch

nv = pytest.importorskip("nvfp4_block_quantization_quantize_gb300")


@pytest.fixture(scope="module")
def lib():
    nv.build()
    return nv.load_library()


# well apart: 2^24 bytes from one to the next, more than any buffer below has
ADDRESS = {n: (i + 1) << 24 for i, n in enumerate(
    ("x", "hidden", "weight", "hidden_out", "out", "codes", "scales", "gamax", "x_scales", "codes_a", "scales_a",
     "offsets", "codes_b", "scales_b", "gamax_a", "gamax_b", "workspace"))}


def at(given, name):
    v = given.get(name, ADDRESS[name])
    return None if v is None else ctypes.c_void_p(v)


M, K = 8, 256


def norm(lib, given, dtype=1, fmt=1, gm=0):
    p = lambda n: at(given, n)                              # noqa: E731
    return lib.nvfp4_rmsnorm(p("x"), p("hidden"), M, K, dtype, p("weight"), 1, 1e-6, p("hidden_out"), p("out"), fmt, gm,
                             p("gamax") if gm else None, 448.0, p("codes"), p("scales"), None)


def mv(lib, given, xt=2, gm=4):
    p = lambda n: at(given, n)                              # noqa: E731
    return lib.nvfp4_mv(p("x"), p("x_scales") if xt == 2 else None, xt, p("codes"), p("scales"), M, 64, K, gm,
                        p("gamax") if gm else None, 448.0, p("out"), 1, None)


def grouped(lib, given, big=False, ga=4):
    p = lambda n: at(given, n)                              # noqa: E731
    E, T, N, k = (8, 8192, 14336, 4096) if big else (4, 8, 64, 64)
    return lib.nvfp4_grouped_mm(p("codes_a"), p("scales_a"), p("offsets"), p("codes_b"), p("scales_b"), E, T, N, k, ga,
                                p("gamax_a"), p("gamax_b"), 448.0, p("out"), 1, p("workspace"), 1 << 40, None)


NORM_OUTS = ("hidden_out", "out", "codes", "scales", "gamax")
NORM_INS = ("x", "hidden", "weight")
SAME = [(a, b) for a in NORM_OUTS for b in NORM_INS + NORM_OUTS if a != b and (a, b) != ("hidden_out", "hidden")]


@pytest.mark.parametrize("output,other", SAME)
def test_norm_output_is_another_buffer(lib, output, other):
    kw = dict(fmt=0, gm=2) if "gamax" in (output, other) else {}
    assert norm(lib, {output: ADDRESS[other]}, **kw) == nv.EINVAL
    assert b"overlap" in lib.nvfp4_last_error()


# bytes of the buffers of norm(): bf16, MXFP8
BYTES = {"x": M * K * 2, "hidden": M * K * 2, "weight": K * 2, "hidden_out": M * K * 2, "out": M * K * 2, "codes": M * K,
         "scales": M * K // 32}


@pytest.mark.parametrize("output", ["hidden_out", "out", "codes", "scales"])
@pytest.mark.parametrize("other", ["x", "hidden", "weight", "out", "codes"])
def test_norm_output_shares_part_of_another(lib, output, other):
    if output == other:
        return
    for shift in (BYTES[other] - 16, -(BYTES[output] - 16)):
        assert norm(lib, {output: ADDRESS[other] + shift}) == nv.EINVAL
        assert b"overlap" in lib.nvfp4_last_error()


def test_norm_in_place_needs_another_x(lib):
    """hidden_out == hidden is the update in place; the x it reads is not that buffer, nor is any other output."""
    for other in ("x", "out", "codes", "scales", "weight"):
        a = ADDRESS["hidden"]
        assert norm(lib, {"hidden_out": a, other: a}) == nv.EINVAL
        assert b"overlap" in lib.nvfp4_last_error()


def test_norm_given_amax_is_not_an_output(lib):
    for gm in (3, 4):
        assert norm(lib, {"codes": ADDRESS["gamax"]}, fmt=0, gm=gm) == nv.EINVAL
        assert b"codes must not overlap gamax" in lib.nvfp4_last_error()


@pytest.mark.parametrize("other", ["x", "x_scales", "codes", "scales", "gamax"])
def test_mv_output_is_an_input(lib, other):
    for shift in (0, -16):
        assert mv(lib, {"out": ADDRESS[other] + shift}) == nv.EINVAL
        assert b"overlap" in lib.nvfp4_last_error()


@pytest.mark.parametrize("other", ["codes_a", "scales_a", "offsets", "codes_b", "scales_b", "gamax_a", "gamax_b"])
def test_grouped_output_is_an_input(lib, other):
    assert grouped(lib, {"out": ADDRESS[other]}) == nv.EINVAL
    assert b"overlap" in lib.nvfp4_last_error()


@pytest.mark.parametrize("other", ["codes_a", "scales_a", "offsets", "codes_b", "scales_b", "gamax_a", "gamax_b", "out"])
def test_grouped_workspace_is_another_buffer(lib, other):
    wide = {n: v << 10 for n, v in ADDRESS.items()}         # apart by 2^34: these buffers are large
    assert grouped(lib, {**wide, "workspace": wide[other]}, big=True) == nv.EINVAL
    assert b"overlap" in lib.nvfp4_last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on addresses that are not")
def test_buffers_side_by_side_are_not_refused(lib):
    """Neighbours that share no byte, and the update in place, pass the checks (and fail at the launch: no device)."""
    side = {"x": 1 << 24}
    for a, b in zip(("x", "hidden", "weight", "hidden_out", "out", "codes"), ("hidden", "weight", "hidden_out", "out", "codes", "scales")):
        side[b] = side[a] + BYTES[a]
    assert norm(lib, side) == nv.ECUDA
    assert norm(lib, {**side, "hidden_out": side["hidden"]}) == nv.ECUDA
    assert norm(lib, {"x": ADDRESS["hidden"]}) == nv.ECUDA  # x and hidden are both read
    assert mv(lib, {}) == nv.ECUDA and grouped(lib, {}) == nv.ECUDA
    assert mv(lib, {"x_scales": ADDRESS["gamax"], "out": ADDRESS["x"] + M * K}) == nv.ECUDA
