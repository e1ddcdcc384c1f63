"""The serving operators at sizes at which a CTA walks: several rows of the norm
(the next row is loaded while the present one is reduced and stored), several row
tiles and rounds of columns of nvfp4_mv (loads run on into the next tile, the
sums' buffers take turns), several token tiles an expert and several blocks of
token tiles of nvfp4_grouped_mm.

References are float64 on the device, written from the formulas.  Where every fp32
partial sum is exact (small integers times scales of 1/2, 1 and 2) the result must
equal them bit for bit; elsewhere the tolerance is the operator's error bound, as in
test_gpu_serving.py.  The sizes are chosen for a GPU of 152 SMs.
"""
import numpy as np
import pytest
import torch

import oracle
from parity_helpers import to_dev

pytestmark = pytest.mark.gpu

nv = pytest.importorskip("nvfp4_block_quantization_quantize_gb300")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    nv.build()
    nv.load_library()


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def unit_weight(gen, *shape):
    """Random codes, scales 1/2, 1 and 2."""
    codes = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = (0x30 + 8 * torch.randint(0, 3, (*shape[:-1], shape[-1] // 16), generator=gen, device="cuda")).to(torch.uint8)
    return codes, scales


def values(codes, scales):
    """float64 values of codes [..., K/2] and scale bytes [..., K/16]."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).int()
    q = grid[c & 7] * (1 - 2 * (c >> 3)).double()
    return q * scales.view(torch.float8_e4m3fn).double().repeat_interleave(16, dim=-1)


def times_weight(x, codes, scales):
    """x W^T in float64, a part of the weight at a time."""
    return torch.cat([x @ values(codes[r:r + 8192], scales[r:r + 8192]).t() for r in range(0, codes.shape[0], 8192)], dim=1)


# ---- nvfp4_mv ---------------------------------------------------------------------------------
MV_WALKS = {
    "tiles of one CTA": (3, 20011, 4096),
    "tiles of one CTA, one token": (1, 40000, 16384),
    "tiles and rounds": (16, 65536, 4096),
    "tiles of a cluster": (16, 8192, 16384),
    "tiles and rounds of a cluster": (16, 16384, 16384),
    "one chunk a warp": (9, 65539, 256),
    "K not of 64, a cluster": (13, 20011, 2064),
    "K not of 64, rounds": (16, 33000, 2064),
    "K not of 64, rounds of a cluster": (16, 12000, 8208),
    "K below a chunk": (7, 70001, 48),
}


@pytest.mark.parametrize("name", sorted(MV_WALKS))
@pytest.mark.parametrize("x_type", ["f32", "bf16", "mxfp8"])
def test_mv_walks(name, x_type):
    M, N, K = MV_WALKS[name]
    gen = generator(M + N + K)
    codes, scales = unit_weight(gen, N, K)
    x = torch.randint(-7, 8, (M, K), generator=gen, device="cuda").float()
    kw = {}
    if x_type == "mxfp8":
        e = torch.randint(0, 2, (M, -(-K // 32)), generator=gen, device="cuda")
        kw["x_scales"] = (127 + e).to(torch.uint8)
        xd = x.to(torch.float8_e4m3fn).view(torch.uint8)
        x = x * torch.pow(2.0, e.float()).repeat_interleave(32, dim=1)[:, :K]
    else:
        xd = x.to(torch.float32 if x_type == "f32" else torch.bfloat16)
    ref = times_weight(x.double(), codes, scales)
    assert float((x.abs().double() @ torch.full((K, 1), 12.0, dtype=torch.float64, device="cuda")).max()) < 2 ** 22
    y = nv.nvfp4_mv(xd, codes, scales, out_dtype="f32", **kw)
    assert torch.equal(y.double(), ref)
    # with one amax a row: the exact sum, one rounding by the row's decode scale
    g = torch.rand(N, generator=gen, device="cuda") * 9 + 0.1
    dec = torch.from_numpy(np.array([oracle.global_scales(float(a), 448.0)[1] for a in g.cpu().numpy()], np.float32)).cuda()
    y = nv.nvfp4_mv(xd, codes, scales, gamax=g, out_dtype="bf16", **kw)
    assert torch.equal(y, (ref.float() * dec).to(torch.bfloat16))


@pytest.mark.parametrize("name", ["tiles of one CTA", "tiles and rounds of a cluster", "K not of 64, rounds"])
def test_mv_walks_on_fp32(name):
    """fp32 activations with all their bits: a chain of 16 products and the fp32 sums after it (2^-22 a step), and
    22 of x's 24 bits (2^-23)."""
    M, N, K = MV_WALKS[name]
    gen = generator(K)
    codes = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.randint(0x28, 0x48, (N, K // 16), generator=gen, device="cuda", dtype=torch.uint8)
    x = torch.randn(M, K, generator=gen, device="cuda")
    y = nv.nvfp4_mv(x, codes, scales, out_dtype="f32").double()
    for r in range(0, N, 8192):
        w = values(codes[r:r + 8192], scales[r:r + 8192])
        bound = (x.double().abs() @ w.abs().t()) * (17 * 2.0 ** -22 + 2.0 ** -23)
        assert bool(((y[:, r:r + 8192] - x.double() @ w.t()).abs() <= bound).all())


# ---- nvfp4_rmsnorm ----------------------------------------------------------------------------
# (rows, K): many more rows than CTAs, at 32 (8 rows a CTA), 96, 128, 256, 512, 544 and 1024 threads a row, and two
# and three passes along a row
NORM_WALKS = [(30011, 512), (13007, 1456), (9001, 2048), (4001, 4096), (2003, 8192), (1501, 8208), (1201, 16384), (801, 16400),
              (701, 40000)]


@pytest.mark.parametrize("M,K", NORM_WALKS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_norm_walks(M, K, dt):
    """Each row of a long call is what it is in a call of few rows (those are checked against the formula and the
    codec elsewhere), bit for bit: out, hidden in place, MXFP8 and NVFP4 codes, amaxes; and out against float64."""
    gen, tdt = generator(K), torch.float32 if dt == "f32" else torch.bfloat16
    x, r = (torch.randn(M, K, generator=gen, device="cuda").to(tdt) for _ in range(2))
    x *= torch.exp(torch.randn(M, 1, generator=gen, device="cuda")).to(tdt)       # rows of their own sizes
    w = 1 + 0.1 * torch.randn(K, generator=gen, device="cuda")
    forms = [dict(want_out=True), dict(format="nvfp4"), dict(format="nvfp4", gamax_mode="row", want_out=True),
             dict(format="nvfp4", gamax_mode="row_given"), dict(want_codes=False, want_out=True)]
    given = torch.rand(M, generator=gen, device="cuda") * 9 + 0.1
    for form in forms:
        h = r.clone()
        kw = dict(form, gamax=given) if form.get("gamax_mode") == "row_given" else form
        got = nv.nvfp4_rmsnorm(x, w, hidden=h, hidden_out=h, eps=1e-5, **kw)
        assert got["hidden"] is h
        for a in range(0, M, 37):
            rows = slice(a, min(a + 37, M))
            if a > 4000 and a + 4000 < M and (a // 37) % 16:                     # all of the first and last, some between
                continue
            kw = dict(form, gamax=given[rows]) if form.get("gamax_mode") == "row_given" else form
            few = nv.nvfp4_rmsnorm(x[rows], w, hidden=r[rows], eps=1e-5, **kw)
            assert set(few) == set(got)
            for k, v in few.items():
                assert torch.equal(got[k][rows], v), (form, k, a)
    h64 = x.double() + r.double()
    y = h64 / torch.sqrt((h64 * h64).mean(dim=1, keepdim=True) + 1e-5) * w.double()
    err = (got["out"].double() - y).abs()
    assert bool((err <= y.abs() * (2.0 ** -17 + (2.0 ** -8 if dt == "bf16" else 0.0)) + 1e-30).all())
    assert torch.equal(got["hidden"], (x.float() + r.float()).to(tdt))


@pytest.mark.parametrize("M,K", [(30011, 512), (4001, 4096), (801, 16400)])
def test_norm_walks_codes(M, K):
    """With float32 in and out a long call's NVFP4 codes are the quantizer's of the norm it returns."""
    gen = generator(M)
    x = torch.randn(M, K, generator=gen, device="cuda")
    got = nv.nvfp4_rmsnorm(x, format="nvfp4", gamax_mode="row", want_out=True)
    q = nv.nvfp4_quantize(got["out"], gamax_mode="row")
    for k in ("codes", "scales", "gamax"):
        assert torch.equal(got[k], q[k]), k


# ---- nvfp4_grouped_mm -------------------------------------------------------------------------
def few_and_one(E, n, large):
    """E groups of n rows, the middle one with `large`."""
    sizes = [n] * E
    sizes[E // 2] = large
    return [0, *np.cumsum(sizes).tolist()]


GROUPED_WALKS = {                                         # experts, offsets, N, K
    "16-token tiles": (40, few_and_one(40, 2, 210), 200, 320),
    "32-token tiles": (24, few_and_one(24, 6, 230), 200, 320),
    "64-token tiles": (16, few_and_one(16, 14, 290), 328, 576),
    "128-token tiles": (7, few_and_one(7, 30, 700), 328, 576),
    "16-token tiles, empty groups": (60, few_and_one(60, 0, 333), 129, 64),
    "blocks of token tiles": (3, [0, 1700, 1701, 5003], 4096, 14336),
    "blocks, rows off the tiles": (5, [0, 900, 2900, 2900, 4111, 5111], 2056, 14400),
    "blocks, many experts": (200, [37 * e + (e > 90) * 1900 for e in range(201)], 1024, 4096),
}


@pytest.mark.parametrize("name", sorted(GROUPED_WALKS))
@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
def test_grouped_walks(name, out_dtype):
    E, offsets, N, K = GROUPED_WALKS[name]
    T = offsets[-1]
    assert (nv.load_library().nvfp4_grouped_mm_workspace(E, T, N, K) > 0) == name.startswith("blocks")
    gen = generator(E + N + K)
    ca, sa = unit_weight(gen, T, K)
    cb, sb = unit_weight(gen, E, N, K)
    y = nv.nvfp4_grouped_mm(ca, sa, torch.tensor(offsets, device="cuda"), cb, nv.nvfp4_grouped_scales_to_mma(sb),
                            out_dtype=out_dtype)
    most = 0.0
    for e in range(E):
        a, b = values(ca[offsets[e]:offsets[e + 1]], sa[offsets[e]:offsets[e + 1]]), values(cb[e], sb[e])
        ref = (a @ b.t()).float()
        if a.shape[0]:
            most = max(most, float((a.abs() @ b.abs().t()).max()))
        assert torch.equal(y[offsets[e]:offsets[e + 1]], ref if out_dtype == "f32" else ref.to(torch.bfloat16)), e
    assert most < 2 ** 20                                 # multiples of 1/16: exact in fp32
