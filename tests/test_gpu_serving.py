"""The serving operators (nvfp4_rmsnorm, nvfp4_mv, nvfp4_grouped_mm) against
plain float64 implementations on the CPU.

Where a case is built so that every fp32 partial sum is exact (unit or
power-of-two scales, small integers) the result must equal the reference bit
for bit; elsewhere the tolerance is the operator's own error bound:
  products   each fp32 accumulation step is off by at most 2^-22 of the sum of
             magnitudes so far (2 ulp: the tensor cores may truncate); nvfp4_mv
             chains at most 16 steps before an fp32 sum, nvfp4_grouped_mm K / 64;
  norm       the sum of squares has at most 100 fp32 roundings in sequence, the
             rest six: 2^-17 of each value.
"""
import numpy as np
import pytest
import torch

import nvfp4_workloads as W
import oracle
from parity_helpers import assert_same, to_dev, to_np

pytestmark = pytest.mark.gpu

nv = pytest.importorskip("nvfp4_block_quantization_quantize_gb300")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    nv.build()
    nv.load_library()


def values(codes, scales, rows, K):
    """float64 values without the global scale."""
    return oracle.dequantize(codes, scales, rows, K, out_dtype=oracle.F32).astype(np.float64)


def decode_scale(gamax, bound=448.0):
    return np.array([oracle.global_scales(float(g), bound)[1] for g in np.ravel(gamax)], np.float64)


def random_weight(rng, N, K, low=0x28, high=0x48):
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    return codes, rng.integers(low, high, (N, K // 16), dtype=np.uint8)


def bf16_round(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).float().numpy()


def e4m3_values(codes):
    return torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn).double().numpy()


# ---- nvfp4_mv ---------------------------------------------------------------------------------
MV_SHAPES = [(1, 1, 16), (1, 16, 32), (2, 17, 48), (3, 128, 64), (5, 33, 528), (8, 129, 1024), (9, 100, 1040),
             (16, 70, 2064), (13, 257, 4096), (4, 2500, 512), (1, 31, 9232), (7, 40, 16384)]


@pytest.mark.parametrize("M,N,K", MV_SHAPES)
@pytest.mark.parametrize("x_type", ["f32", "bf16", "mxfp8"])
def test_mv_exact(M, N, K, x_type):
    """Integers times unit-scale codes: every partial sum is a multiple of 1/4 below 2^22."""
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    scales = (0x38 + 8 * rng.integers(-1, 2, (N, K // 16))).astype(np.uint8)     # 1/2, 1, 2
    x = rng.integers(-7, 8, (M, K)).astype(np.float32)
    kw = {}
    if x_type == "mxfp8":
        e = rng.integers(0, 2, (M, -(-K // 32)))
        xd = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
        kw["x_scales"] = torch.from_numpy((127 + e).astype(np.uint8)).cuda()
        x = x * np.repeat(2.0 ** e, 32, axis=1)[:, :K]
    else:
        xd = torch.from_numpy(x).cuda().to(torch.float32 if x_type == "f32" else torch.bfloat16)
    y = nv.nvfp4_mv(xd, to_dev(codes), to_dev(scales), out_dtype="f32", **kw)
    ref = x.astype(np.float64) @ values(codes, scales, N, K).T
    assert np.abs(ref).max() < 2 ** 22
    assert np.array_equal(to_np(y).astype(np.float64), ref)


@pytest.mark.parametrize("M,N,K", [(1, 1000, 4096), (6, 300, 2064), (16, 130, 7168)])
@pytest.mark.parametrize("x_type", ["f32", "bf16"])
@pytest.mark.parametrize("gm", ["none", "tensor", "row"])
@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
def test_mv_quantized_weight(M, N, K, x_type, gm, out_dtype):
    w = W.matrix((N, K), seed=N + K, dtype="f32", dist="t")
    x = W.matrix((M, K), seed=M, dtype=x_type, dist="t")
    q = nv.nvfp4_quantize(to_dev(w), gamax_mode=gm)
    y = nv.nvfp4_mv(to_dev(x), q["codes"], q["scales"], gamax=q.get("gamax"), out_dtype=out_dtype)
    wv = values(to_np(q["codes"]), to_np(q["scales"]), N, K)
    if gm != "none":
        wv = wv * decode_scale(to_np(q["gamax"]))[:, None]
    xv = (W.bf16_bits_to_f32(x) if x_type == "bf16" else x).astype(np.float64)
    ref = xv @ wv.T
    bound = (np.abs(xv) @ np.abs(wv).T) * (16 * 2.0 ** -22 + 2.0 ** -22)
    if out_dtype == "bf16":
        bound = bound + np.abs(ref) * 2.0 ** -8
    assert y.shape == (M, N) and (np.abs(to_np(y.float()).astype(np.float64) - ref) <= bound + 1e-30).all()


def test_mv_takes_the_norm_output():
    x = to_dev(W.matrix((5, 4112), seed=3, dtype="bf16", dist="t"))
    w = to_dev(W.matrix((77, 4112), seed=5, dtype="bf16"))
    q, n = nv.nvfp4_quantize(w), nv.nvfp4_rmsnorm(x)
    y = nv.nvfp4_mv(n["codes"], q["codes"], q["scales"], x_scales=n["scales"], out_dtype="f32")
    y2 = nv.nvfp4_mv(n["codes"].view(torch.float8_e4m3fn), q["codes"], q["scales"],
                     x_scales=n["scales"].view(torch.float8_e8m0fnu), out_dtype="f32")
    assert torch.equal(y, y2)
    xv = e4m3_values(to_np(n["codes"])) * np.repeat(2.0 ** (to_np(n["scales"]).astype(np.float64) - 127), 32, 1)[:, :4112]
    wv = values(to_np(q["codes"]), to_np(q["scales"]), 77, 4112)
    assert (np.abs(to_np(y) - xv @ wv.T) <= (np.abs(xv) @ np.abs(wv).T) * 2.0 ** -17).all()


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1.0, 1e30])
@pytest.mark.parametrize("x_type", ["f32", "bf16"])
def test_mv_range(scale, x_type):
    """Far magnitudes, and a token whose slices differ by 2^100."""
    rng = np.random.default_rng(7)
    M, N, K = 3, 40, 2048
    codes, scales = random_weight(rng, N, K)
    x = rng.standard_normal((M, K)) * scale
    x[1, :1024] *= 2.0 ** (-100 if scale >= 1 else 100)
    x[2, 5:] = 0.0
    xd = torch.from_numpy(x.astype(np.float32)).cuda()
    xd = xd if x_type == "f32" else xd.to(torch.bfloat16)
    xv = xd.double().cpu().numpy()
    y = to_np(nv.nvfp4_mv(xd, to_dev(codes), to_dev(scales), out_dtype="f32")).astype(np.float64)
    wv = values(codes, scales, N, K)
    # besides the sums: what lies 2^39 below a slice's maximum, and fp32's own subnormals
    lost = np.repeat(np.abs(xv).reshape(M, 2, 1024).max(2) * 2.0 ** -39, 1024, axis=1)
    bound = (np.abs(xv) @ np.abs(wv).T) * 2.0 ** -17 + lost @ np.abs(wv).T + K * 2.0 ** -149
    assert (np.abs(y - xv @ wv.T) <= bound).all()


@pytest.mark.parametrize("zero_scale", [0, 127, 254, 255])
@pytest.mark.parametrize("M,K", [(1, 512), (5, 2064)])
def test_mv_mxfp8_zero_groups(zero_scale, M, K):
    """A group of zeros may have any scale: it takes no range from the small ones (NaN: the row is NaN)."""
    rng = np.random.default_rng(K + zero_scale)
    N, groups = 50, -(-K // 32)
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    scales = (0x38 + 8 * rng.integers(-1, 2, (N, K // 16))).astype(np.uint8)
    x = rng.integers(-7, 8, (M, K)).astype(np.float32)
    b = np.full((M, groups), 127 - 60, np.uint8)
    zero = rng.random((M, groups)) < 0.4
    zero[0] = True                                        # a token of zeros alone
    zero[:, -1] = True
    b[zero] = zero_scale
    x[np.repeat(zero, 32, axis=1)[:, :K]] = 0.0
    xd = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8)
    xd[torch.from_numpy(x == 0)] = torch.from_numpy((rng.integers(0, 2, int((x == 0).sum())) * 128).astype(np.uint8))      # either zero
    y = to_np(nv.nvfp4_mv(xd.cuda(), to_dev(codes), to_dev(scales), x_scales=to_dev(b), out_dtype="f32"))
    if zero_scale == 255:
        assert np.isnan(y).all()
        return
    ref = (x.astype(np.float64) * 2.0 ** -60) @ values(codes, scales, N, K).T
    assert np.array_equal(y.astype(np.float64), ref) and (M == 1 or np.abs(ref[1:]).max() > 0)


def test_mv_special_values():
    """NaN and infinities of x reach every product they take part in and no other token."""
    rng = np.random.default_rng(11)
    M, N, K = 4, 33, 1056
    codes, scales = random_weight(rng, N, K)
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[1, 7] = np.nan
    x[2, 1030] = np.inf
    for dt in (torch.float32, torch.bfloat16):
        xd = torch.from_numpy(x).cuda().to(dt)
        y = to_np(nv.nvfp4_mv(xd, to_dev(codes), to_dev(scales), out_dtype="f32"))
        clean = xd.clone()
        clean[1:3] = 0.0
        c = to_np(nv.nvfp4_mv(clean, to_dev(codes), to_dev(scales), out_dtype="f32"))
        assert np.isnan(y[1]).all()
        assert np.array_equal(y[[0, 3]], c[[0, 3]])
        w = values(codes, scales, N, K)[:, 1030]
        want = np.where(w == 0, np.nan, np.sign(w) * np.inf)
        assert np.array_equal(y[2], want.astype(np.float32), equal_nan=True)


def test_mv_same_bits_each_run():
    q = nv.nvfp4_quantize(to_dev(W.matrix((600, 9216), seed=1, dtype="bf16")))
    x = to_dev(W.matrix((16, 9216), seed=2, dtype="f32"))
    y = nv.nvfp4_mv(x, q["codes"], q["scales"], out_dtype="f32")
    for _ in range(5):
        assert torch.equal(y, nv.nvfp4_mv(x, q["codes"], q["scales"], out_dtype="f32"))


def test_mv_empty_strided_and_out():
    q = nv.nvfp4_quantize(to_dev(W.matrix((48, 64), seed=1, dtype="bf16")))
    x = to_dev(W.matrix((6, 128), seed=2, dtype="bf16"))
    assert nv.nvfp4_mv(x[:0, :64].contiguous(), q["codes"], q["scales"]).shape == (0, 48)
    assert nv.nvfp4_mv(x[:, :64].contiguous(), q["codes"][:0], q["scales"][:0]).shape == (6, 0)
    e = torch.empty((3, 0), device="cuda")
    z = nv.nvfp4_mv(e, torch.empty((5, 0), dtype=torch.uint8, device="cuda"),
                    torch.empty((5, 0), dtype=torch.uint8, device="cuda"), out_dtype="f32")
    assert torch.equal(z, torch.zeros((3, 5), device="cuda"))
    half = x[:, :64]                                      # strided rows
    y = nv.nvfp4_mv(half, q["codes"], q["scales"])
    assert torch.equal(y, nv.nvfp4_mv(half.contiguous(), q["codes"], q["scales"]))
    buf = torch.full((8, 48), 7.0, device="cuda", dtype=torch.bfloat16)
    nv.nvfp4_mv(half, q["codes"], q["scales"], out=buf[1:7])
    assert torch.equal(buf[1:7], y) and bool((buf[0] == 7).all()) and bool((buf[7] == 7).all())


# ---- nvfp4_rmsnorm ----------------------------------------------------------------------------
def norm_reference(x, hidden, weight, eps):
    h = x.astype(np.float64) + (0 if hidden is None else hidden.astype(np.float64))
    y = h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    return h, y if weight is None else y * weight.astype(np.float64)


def mxfp8_of(y):
    """MXFP8 of float32 y as the header defines it, finite y: (codes, scales)."""
    M, K = y.shape
    p = np.zeros((M, -(-K // 32) * 32), np.float32)
    p[:, :K] = y
    p = p.reshape(M, -1, 32)
    m, k = np.frexp(np.abs(p).max(axis=2))
    e = np.where(m == 0, -127, np.maximum(np.where(m > 0.875, k - 8, k - 9), -127))
    v = np.ldexp(p.astype(np.float64), -e[..., None]).astype(np.float32)
    c = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy().reshape(M, -1)[:, :K]
    return np.ascontiguousarray(c), (e + 127).astype(np.uint8)


NORM_SHAPES = [(1, 16), (3, 48), (2, 512), (5, 1040), (1, 4096), (33, 4096), (4, 8208), (2, 16384), (3, 16400),
               (2, 40000)]


@pytest.mark.parametrize("M,K", NORM_SHAPES)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("add", [False, True])
def test_norm_values(M, K, dt, add):
    x = W.matrix((M, K), seed=K + M, dtype=dt, dist="t")
    r = W.matrix((M, K), seed=K + M + 1, dtype=dt) if add else None
    w = W.matrix((1, K), seed=9, dtype="f32")[0]
    f = W.bf16_bits_to_f32 if dt == "bf16" else (lambda v: v)
    got = nv.nvfp4_rmsnorm(to_dev(x), to_dev(w), hidden=None if r is None else to_dev(r), eps=1e-5, want_out=True)
    h, y = norm_reference(f(x), None if r is None else f(r), w, 1e-5)
    out = to_np(got["out"].float()).astype(np.float64)
    assert (np.abs(out - y) <= np.abs(y) * (2.0 ** -17 + (2.0 ** -8 if dt == "bf16" else 0.0)) + 1e-30).all()
    if add:                                               # one fp32 addition, one rounding to the type
        want = (f(x) + f(r)).astype(np.float32)
        assert_same(to_np(got["hidden"].float()), bf16_round(want) if dt == "bf16" else want, "hidden")
    # the dequantized output is within half an E4M3 step (2^-4 of the value, 2^-10 of the scale at the least)
    s = np.repeat(2.0 ** (to_np(got["scales"]).astype(np.float64) - 127), 32, axis=1)[:, :K]
    q = e4m3_values(to_np(got["codes"])) * s
    assert (np.abs(q - y) <= np.maximum(np.abs(y) * 2.0 ** -4, s * 2.0 ** -10) * 1.0001 + np.abs(y) * 2.0 ** -17).all()
    # and no scale is larger than needed, nor too small
    top = np.zeros((M, s.shape[1] + (-K) % 32))
    top[:, :K] = np.abs(y)
    top = top.reshape(M, -1, 32).max(axis=2)
    sc = 2.0 ** (to_np(got["scales"]).astype(np.float64) - 127)
    assert (top <= 448 * sc * (1 + 2.0 ** -17)).all() and ((top >= 224 * sc * (1 - 2.0 ** -17)) | (top == 0)).all()


@pytest.mark.parametrize("M,K", [(7, 48), (2, 4112), (3, 16400), (2, 40000)])
def test_norm_codes_are_those_of_its_output(M, K):
    """With float32 in and out, the codes are bit for bit the quantization of the
    norm the call also returns; bfloat16 input gives the codes of its float32 copy."""
    x, r = W.matrix((M, K), seed=1, dtype="bf16", dist="t"), W.matrix((M, K), seed=2, dtype="bf16")
    w = W.matrix((1, K), seed=3, dtype="bf16")[0]
    xd, rd, wd = to_dev(x), to_dev(r), to_dev(w)
    got = nv.nvfp4_rmsnorm(xd.float(), wd, hidden=rd.float(), want_out=True)
    c, s = mxfp8_of(to_np(got["out"]))
    assert_same(to_np(got["codes"]), c, "mxfp8 codes")
    assert_same(to_np(got["scales"]), s, "mxfp8 scales")
    low = nv.nvfp4_rmsnorm(xd, wd.float(), hidden=rd)
    assert_same(to_np(low["codes"]), c, "bf16 codes")
    for gm, ogm in (("none", oracle.GAMAX_NONE), ("row", oracle.GAMAX_ROW), ("tensor_given", oracle.GAMAX_TENSOR_GIVEN),
                    ("row_given", oracle.GAMAX_ROW_GIVEN)):
        kw, okw = {}, {}
        if gm.endswith("given"):
            A = np.linspace(3.0, 9.0, M if gm == "row_given" else 1).astype(np.float32)
            kw["gamax"], okw["gamax"] = to_dev(A), A
        g = nv.nvfp4_rmsnorm(xd.float(), wd, hidden=rd.float(), format="nvfp4", gamax_mode=gm, want_out=True, **kw)
        o = oracle.quantize(to_np(g["out"]), gamax_mode=ogm, **okw)
        assert_same(to_np(g["codes"]), o["codes"], gm)
        assert_same(to_np(g["scales"]), o["scales"], gm)
        if gm == "row":
            assert_same(to_np(g["gamax"]), o["gamax"], "row amax")


def test_norm_in_place_and_without_codes():
    x, r = to_dev(W.matrix((9, 256), seed=1, dtype="bf16")), to_dev(W.matrix((9, 256), seed=2, dtype="bf16"))
    a = nv.nvfp4_rmsnorm(x, hidden=r, want_out=True)
    r2 = r.clone()
    b = nv.nvfp4_rmsnorm(x, hidden=r2, hidden_out=r2, want_codes=False, want_out=True)
    assert set(b) == {"hidden", "out"} and b["hidden"] is r2
    assert torch.equal(r2, a["hidden"]) and torch.equal(b["out"], a["out"])
    s = nv.nvfp4_rmsnorm(torch.cat([x, x], 1)[:, :256], hidden=torch.cat([r, r], 1)[:, 256:])     # strided rows
    assert torch.equal(s["codes"], a["codes"]) and torch.equal(s["hidden"], a["hidden"])


def test_norm_special_values():
    x = np.zeros((6, 96), np.float32)
    x[1] = 1e-30                                          # squares below fp32's range
    x[2] = 1e25                                           # squares past it
    x[3, :] = 1.0
    x[3, 40] = np.nan
    x[4, :] = 1.0
    x[4, 3] = np.inf
    x[5, 0] = 1.0
    for dt in (torch.float32, torch.bfloat16):
        got = nv.nvfp4_rmsnorm(torch.from_numpy(x).cuda().to(dt), want_out=True)
        out, c, s = to_np(got["out"].float()), to_np(got["codes"]), to_np(got["scales"])
        assert (out[0] == 0).all() and (c[0] == 0).all() and (s[0] == 0).all()
        assert np.allclose(out[1], 1e-27, rtol=1e-2, atol=0) and (np.abs(e4m3_values(c[1])) <= 448).all()
        assert (out[2] == 0).all() and (c[2] == 0).all()
        assert np.isnan(out[3]).all() and (c[3] & 0x7F == 0x7F).all()
        assert np.isnan(out[4, 3]) and (np.delete(out[4], 3) == 0).all()
        assert c[4, 3] & 0x7F == 0x7F and (np.delete(c[4], 3) & 0x7F == 0).all()
        want = np.sqrt(96.0)                              # 1 / sqrt(1 / 96 + 1e-6)
        assert abs(out[5, 0] / want - 1) < 1e-2 and (out[5, 1:] == 0).all()


def test_norm_empty():
    for M, K in ((0, 64), (4, 0)):
        got = nv.nvfp4_rmsnorm(torch.empty((M, K), device="cuda"))
        assert got["codes"].shape == (M, K)
    g = nv.nvfp4_rmsnorm(torch.empty((4, 0), device="cuda"), format="nvfp4", gamax_mode="row")
    assert to_np(g["gamax"]).tolist() == [0.0] * 4


# ---- nvfp4_grouped_mm -------------------------------------------------------------------------
def grouped_reference(ca, sa, cb, sb, offsets, K, ga=None, gb=None):
    T, (E, N) = ca.shape[0], cb.shape[:2]
    A = values(ca, sa, T, K)
    y, mag = np.zeros((T, N)), np.zeros((T, N))
    for e in range(E):
        r = slice(offsets[e], offsets[e + 1])
        B = values(cb[e], sb[e], N, K)
        d = 1.0 if gb is None else decode_scale(gb[e])
        y[r], mag[r] = (A[r] @ B.T) * d, (np.abs(A[r]) @ np.abs(B).T) * d
    if ga is not None:
        d = decode_scale(ga)[:, None]
        y, mag = y * d, mag * d
    return y, mag


def grouped_inputs(rng, E, T, N, K, scales=None):
    low, high = (0x28, 0x48) if scales is None else scales
    ca, sa = random_weight(rng, T, K, low, high)
    cb, sb = random_weight(rng, E * N, K, low, high)
    return ca, sa, cb.reshape(E, N, K // 2), sb.reshape(E, N, K // 16)


def grouped_gpu(ca, sa, offsets, cb, sb, **kw):
    off = torch.tensor(offsets, dtype=torch.int64, device="cuda")
    return nv.nvfp4_grouped_mm(to_dev(ca), to_dev(sa), off, to_dev(cb), nv.nvfp4_grouped_scales_to_mma(to_dev(sb)), **kw)


GROUPS = {
    "one token": (1, [0, 1]),
    "two of five": (5, [0, 0, 1, 1, 2, 2]),
    "ragged": (6, [0, 3, 3, 20, 21, 100, 117]),
    "first and last empty": (4, [0, 0, 64, 128, 128]),
    "one expert takes all": (3, [0, 0, 300, 300]),
    "exact tiles": (2, [0, 128, 256]),
    "past a tile": (2, [0, 129, 258]),
    "many experts": (40, list(range(41))),
    "large": (2, [0, 700, 1100]),
}


@pytest.mark.parametrize("name", sorted(GROUPS))
@pytest.mark.parametrize("N,K", [(128, 64), (200, 320), (1, 256), (384, 1088)])
def test_grouped_exact(name, N, K):
    """Scales 1/2, 1 and 2: every partial sum is exact in fp32."""
    E, offsets = GROUPS[name]
    rng = np.random.default_rng(E + N + K)
    ca, sa, cb, sb = grouped_inputs(rng, E, offsets[-1], N, K)
    sa = (0x38 + 8 * rng.integers(-1, 2, sa.shape)).astype(np.uint8)
    sb = (0x38 + 8 * rng.integers(-1, 2, sb.shape)).astype(np.uint8)
    y = grouped_gpu(ca, sa, offsets, cb, sb, out_dtype="f32")
    ref, mag = grouped_reference(ca, sa, cb, sb, offsets, K)
    assert mag.max() < 2 ** 20                            # multiples of 1/16 below 2^20
    assert np.array_equal(to_np(y).astype(np.float64), ref)


def values_on_device(codes, scales):
    """float64 values of codes [..., K/2] and scale bytes [..., K/16] on the device (large cases)."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).int()
    q = grid[c & 7] * (1 - 2 * (c >> 3)).double()
    return q * scales.view(torch.float8_e4m3fn).double().repeat_interleave(16, dim=-1)


def grouped_reference_on_device(ca, sa, cb, sb, offsets):
    A = values_on_device(to_dev(ca), to_dev(sa))
    y, mag = [], []
    for e in range(cb.shape[0]):
        a, B = A[offsets[e]:offsets[e + 1]], values_on_device(to_dev(cb[e]), to_dev(sb[e]))
        y.append(a @ B.t())
        mag.append(a.abs() @ B.abs().t())
    return torch.cat(y), torch.cat(mag)


PAIRS = {                                                 # many tokens an expert: pairs of SMs
    "ragged": (4, [0, 1000, 1000, 1033, 2500], 4096, 4160),
    "rows off the tiles": (3, [0, 191, 900, 1733], 6008, 4160),
    "N not of 8": (2, [0, 769, 1600], 6001, 4160),
    "one expert": (1, [0, 1536], 6144, 4224),
    "second half past N": (2, [0, 1000, 2000], 6272, 4160),
    "many tiles": (1, [0, 960], 20000, 2112),
    "whole stages": (1, [0, 1536], 6144, 4096),
    "half a stage at the end": (3, [0, 700, 900, 2000], 4096, 4352),
    "a ragged second half": (3, [0, 700, 900, 2000], 4096, 4416),
    "over 256 experts": (257, list(range(0, 257 * 250 + 1, 250)), 512, 1088),
}


@pytest.mark.parametrize("name", sorted(PAIRS))
@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
def test_grouped_pairs_exact(name, out_dtype):
    E, offsets, N, K = PAIRS[name]
    T = offsets[-1]
    assert nv.load_library().nvfp4_grouped_mm_workspace(E, T, N, K) > 0
    rng = np.random.default_rng(E + N + K)
    ca, sa, cb, sb = grouped_inputs(rng, E, T, N, K)
    sa = (0x38 + 8 * rng.integers(-1, 2, sa.shape, dtype=np.int8)).astype(np.uint8)
    sb = (0x38 + 8 * rng.integers(-1, 2, sb.shape, dtype=np.int8)).astype(np.uint8)
    y = grouped_gpu(ca, sa, offsets, cb, sb, out_dtype=out_dtype)
    ref, mag = grouped_reference_on_device(ca, sa, cb, sb, offsets)
    assert float(mag.max()) < 2 ** 20                     # multiples of 1/16: exact in fp32
    assert torch.equal(y, ref.float() if out_dtype == "f32" else ref.float().to(torch.bfloat16))


def test_grouped_pairs_scales_and_rows_in_no_group():
    rng = np.random.default_rng(15)
    E, offsets, N, K, T = 3, [5, 905, 905, 2105], 4104, 4224, 2200
    assert nv.load_library().nvfp4_grouped_mm_workspace(E, T, N, K) > 0
    ca, sa, cb, sb = grouped_inputs(rng, E, T, N, K)
    sa[:5] = sa[2105:] = 0x7F
    ga, gb = rng.uniform(0.1, 9.0, T).astype(np.float32), rng.uniform(0.1, 9.0, E).astype(np.float32)
    buf = torch.full((T, N), 5.0, device="cuda")
    y = grouped_gpu(ca, sa, offsets, cb, sb, out_dtype="f32", out=buf, gamax_a=to_dev(ga), gamax_b=to_dev(gb))
    assert bool((y[:5] == 5).all()) and bool((y[2105:] == 5).all())
    ref, mag = grouped_reference_on_device(ca[5:2105], sa[5:2105], cb, sb, [0, 900, 900, 2100])
    d = torch.from_numpy(decode_scale(ga[5:2105])).cuda()[:, None]
    g = torch.from_numpy(decode_scale(gb)).cuda()
    d = d * torch.cat([g[0].repeat(900), g[2].repeat(1200)])[:, None]
    assert bool(((y[5:2105].double() - ref * d).abs() <= mag * d * (K / 64 + 4) * 2.0 ** -22).all())


@pytest.mark.parametrize("a_mode", ["none", "tensor", "row"])
@pytest.mark.parametrize("b_amax", [False, True])
@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
def test_grouped_global_scales(a_mode, b_amax, out_dtype):
    rng = np.random.default_rng(5)
    E, offsets, N, K = 5, [0, 7, 7, 150, 151, 400], 257, 704
    T = offsets[-1]
    ca, sa, cb, sb = grouped_inputs(rng, E, T, N, K)
    ga = {"none": None, "tensor": np.float32([2.5]), "row": rng.uniform(0.1, 9.0, T).astype(np.float32)}[a_mode]
    gb = rng.uniform(0.1, 9.0, E).astype(np.float32) if b_amax else None
    if a_mode == "row":
        ga[3], ga[9] = 0.0, np.inf                        # no positive finite amax: scale 1
    y = grouped_gpu(ca, sa, offsets, cb, sb, out_dtype=out_dtype, gamax_a=None if ga is None else to_dev(ga),
                    gamax_b=None if gb is None else to_dev(gb))
    ref, mag = grouped_reference(ca, sa, cb, sb, offsets, K, ga, gb)
    bound = mag * (K / 64 + 4) * 2.0 ** -22 + (np.abs(ref) * 2.0 ** -8 if out_dtype == "bf16" else 0.0)
    assert (np.abs(to_np(y.float()).astype(np.float64) - ref) <= bound).all()


def test_grouped_rows_in_no_group_stay():
    rng = np.random.default_rng(8)
    E, offsets, N, K, T = 3, [4, 9, 9, 30], 72, 128, 37
    ca, sa, cb, sb = grouped_inputs(rng, E, T, N, K)
    sa[30:] = 0x7F                                        # NaN scales in rows of no group
    sa[:4] = 0x7F
    buf = torch.full((T, N), 5.0, device="cuda")
    y = to_np(grouped_gpu(ca, sa, offsets, cb, sb, out_dtype="f32", out=buf))
    ref, mag = grouped_reference(ca[4:30], sa[4:30], cb, sb, [0, 5, 5, 26], K)
    assert (y[:4] == 5).all() and (y[30:] == 5).all()
    assert (np.abs(y[4:30] - ref) <= mag * 2.0 ** -19).all()


def test_grouped_neighbours_and_nan():
    """A NaN scale in a row stays in that row, in its own group and past its end."""
    rng = np.random.default_rng(9)
    E, offsets, N, K = 3, [0, 5, 21, 40], 130, 192
    ca, sa, cb, sb = grouped_inputs(rng, E, 40, N, K)
    clean = to_np(grouped_gpu(ca, sa, offsets, cb, sb, out_dtype="f32"))
    sa2 = sa.copy()
    sa2[5, 0] = sa2[12, 3] = 0x7F
    y = to_np(grouped_gpu(ca, sa2, offsets, cb, sb, out_dtype="f32"))
    rest = [i for i in range(40) if i not in (5, 12)]
    assert np.isnan(y[[5, 12]]).all() and np.array_equal(y[rest], clean[rest])


def test_grouped_offsets_outside_are_clamped():
    rng = np.random.default_rng(10)
    E, N, K, T = 3, 64, 64, 20
    ca, sa, cb, sb = grouped_inputs(rng, E, T, N, K)
    good = grouped_gpu(ca, sa, [0, 8, 8, 20], cb, sb, out_dtype="f32")
    y = grouped_gpu(ca, sa, [-(1 << 40), 8, 8, 1 << 40], cb, sb, out_dtype="f32")
    assert torch.equal(y, good)


def test_grouped_empty():
    rng = np.random.default_rng(12)
    ca, sa, cb, sb = grouped_inputs(rng, 2, 3, 32, 64)
    assert grouped_gpu(ca[:0], sa[:0], [0, 0, 0], cb, sb).shape == (0, 32)
    assert grouped_gpu(ca, sa, [0, 1, 3], cb[:, :0], sb[:, :0]).shape == (3, 0)
    z = torch.full((3, 32), 9.0, device="cuda")
    e8 = torch.uint8
    nv.nvfp4_grouped_mm(torch.empty((3, 0), dtype=e8, device="cuda"), torch.empty((3, 0), dtype=e8, device="cuda"),
                        torch.tensor([0, 1, 2], device="cuda"), torch.empty((2, 32, 0), dtype=e8, device="cuda"),
                        torch.empty((2, 128, 0), dtype=e8, device="cuda"), out=z, out_dtype="f32")
    assert bool((z[:2] == 0).all()) and bool((z[2] == 9).all())


def test_grouped_equals_the_plain_product():
    """One expert and whole tiles: nvfp4_mm's bits."""
    rng = np.random.default_rng(13)
    T, N, K = 256, 384, 1024
    ca, sa, cb, sb = grouped_inputs(rng, 1, T, N, K)
    y = grouped_gpu(ca, sa, [0, T], cb, sb, out_dtype="f32")
    m = nv.nvfp4_mm(to_dev(ca), nv.nvfp4_scales_to_mma(to_dev(sa)), to_dev(cb[0]), nv.nvfp4_scales_to_mma(to_dev(sb[0])),
                    T, N, K, out_dtype="f32")
    ref, mag = grouped_reference(ca, sa, cb, sb, [0, T], K)
    assert (np.abs(to_np(y) - to_np(m)) <= mag * 2 * (K / 64) * 2.0 ** -22).all()


# ---- streams ----------------------------------------------------------------------------------
def test_calls_on_another_stream():
    x = to_dev(W.matrix((4, 512), seed=1, dtype="bf16"))
    q = nv.nvfp4_quantize(to_dev(W.matrix((96, 512), seed=2, dtype="bf16")))
    want = nv.nvfp4_mv(x, q["codes"], q["scales"])
    n = nv.nvfp4_rmsnorm(x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for st in (s, s.cuda_stream, 0):
        y = nv.nvfp4_mv(x, q["codes"], q["scales"], stream=st)
        m = nv.nvfp4_rmsnorm(x, stream=st)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(m["codes"], n["codes"])


def test_chain_in_a_cuda_graph():
    x, r = to_dev(W.matrix((2, 1024), seed=1, dtype="bf16")), to_dev(W.matrix((2, 1024), seed=2, dtype="bf16"))
    q = nv.nvfp4_quantize(to_dev(W.matrix((512, 1024), seed=3, dtype="bf16")))

    def step():
        n = nv.nvfp4_rmsnorm(x, hidden=r)
        return nv.nvfp4_mv(n["codes"], q["codes"], q["scales"], x_scales=n["scales"])

    want = step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = step()
    y.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


# ---- refusals of the binding ------------------------------------------------------------------
def test_binding_refuses_mismatched_tensors():
    q = nv.nvfp4_quantize(to_dev(W.matrix((128, 128), seed=1, dtype="bf16")))
    x = torch.zeros((4, 128), device="cuda", dtype=torch.bfloat16)
    c, s = q["codes"], q["scales"]
    bad = [dict(codes=c[:, :32]), dict(scales=s[:64]), dict(codes=c.to(torch.int8)), dict(x=x.half()),
           dict(gamax=torch.ones(3, device="cuda")), dict(gamax=torch.ones(1)), dict(codes=c.cpu()),
           dict(out=torch.empty((4, 127), device="cuda", dtype=torch.bfloat16)),
           dict(out=torch.empty((4, 128), device="cuda")), dict(x_scales=torch.zeros((4, 4), device="cuda"))]
    for kw in bad:
        args = dict(x=x, codes=c, scales=s)
        args.update(kw)
        with pytest.raises((ValueError, TypeError)):
            nv.nvfp4_mv(**args)
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_mv(torch.zeros((17, 128), device="cuda"), c, s)
    for kw in (dict(weight=torch.ones(64, device="cuda")), dict(weight=torch.ones(128)), dict(hidden=x.float()),
               dict(hidden=x[:2]), dict(hidden_out=x), dict(codes=torch.empty((4, 64), device="cuda", dtype=torch.uint8)),
               dict(format="fp6"), dict(out=x.float())):
        with pytest.raises((ValueError, TypeError)):
            nv.nvfp4_rmsnorm(x, **kw)
    off = torch.tensor([0, 128], device="cuda")
    m = nv.nvfp4_grouped_scales_to_mma(s[None])
    assert torch.equal(m[0], nv.nvfp4_scales_to_mma(s))
    for kw in (dict(offsets=off.int()), dict(offsets=off[:1]), dict(offsets=off.cpu()), dict(scales_b=s[None]),
               dict(codes_b=c), dict(gamax_b=torch.ones(2, device="cuda")), dict(scales_a=s[:4]),
               dict(gamax_a=torch.ones(5, device="cuda"))):
        args = dict(codes_a=c, scales_a=s, offsets=off, codes_b=c[None], scales_b=m)
        args.update(kw)
        if kw.keys() == {"scales_b"}:                     # 128 rows of 8 columns: the same bytes, so use 1 more row
            args["codes_b"] = torch.cat([c, c[:1]])[None]
        with pytest.raises((ValueError, TypeError)):
            nv.nvfp4_grouped_mm(**args)
