"""Attention whose first key takes nearly all weight and has no value, so that the output is made of small weights alone:
they keep their bits, however the kernels hold them on their way into the second product."""
import pytest
import torch

from cache_helpers import attention, parts, take, tolerance, values

nv = pytest.importorskip("nvfp4_block_quantization_quantize_gb300")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def check(x, n, Hq, H, D, L, gap, floor):
    """n queries on L keys, the first of which stands `gap` above the others' logits; no mask.  `floor`: half a step of the
    smallest weights, in parts of the largest: what a kernel may leave out of each key."""
    g = torch.Generator(device="cuda").manual_seed(7)
    P = 16
    pages = -(-L // P)
    cache = nv.nvfp4_cache_empty(pages, P, H, D)
    k, v = torch.zeros(L, H, D, device="cuda"), torch.randn(L, H, D, generator=g, device="cuda").abs()
    k[0, :, 0], v[0] = 6.0, 0.0
    k[:, :, 1] = torch.rand(L, H, generator=g, device="cuda").round()      # the others' logits are not all alike
    j = torch.arange(L, device="cuda")
    nv.nvfp4_cache_write(cache, k, v, j)
    q = torch.zeros(n, Hq, D, device="cuda")
    q[..., 0] = gap / 6.0 + 0.3 * torch.rand(n, Hq, generator=g, device="cuda")
    q[..., 1] = 0.7
    q = q.to(DT[x])
    got, lse = nv.nvfp4_cache_attention(q, cache, j[:pages].int().view(1, -1), torch.tensor([L], device="cuda"), scale=1.0,
                                        offsets=torch.tensor([0, n], device="cuda"), causal=False, out_dtype="f32", want_lse=True)
    kc, ks, vc, vs = (take(p, j) for p in parts(cache))
    kk, vv = values(kc, ks), values(vc, vs)
    assert (vv[0] == 0).all()
    out, want, mass, most = attention(q, kk, vv, n, scale=1.0, causal=False)
    tol = tolerance(out, mass, most, 0.0, L, D, q.dtype, got.dtype) + L * floor * vv.abs().max().item()
    assert (tol < 0.5 * out).all()                         # (a kernel that drops these weights fails)
    off = (got.double() - out).abs()
    assert (off <= tol).all(), (off / out).max().item()
    assert ((lse.double() - want).abs() <= (D + 8) * 2.0 ** -23 * most + 2.0 ** -22 * want.abs() + (L / 16 + 64) * 2.0 ** -23).all()


SHAPES = [(1, 4, 2, 128, 1000), (1, 8, 1, 64, 700), (3, 4, 4, 256, 900), (1, 6, 2, 128, 6000), (2, 24, 2, 128, 1500)]


@pytest.mark.parametrize("gap", [9.0, 15.0, 18.0, 20.0])
@pytest.mark.parametrize("shape", SHAPES)
def test_bf16_queries(shape, gap):
    """A weight as one f16, the largest at 2^11 or above when the reference is set: half a step of 2^-25 is 2^-36 of it."""
    n, Hq, H, D, L = shape
    check("bf16", n, Hq, H, D, L, gap, 2.0 ** -36)


@pytest.mark.parametrize("gap", [9.0, 15.0, 18.0, 24.0])
@pytest.mark.parametrize("shape", SHAPES)
def test_fp32_queries(shape, gap):
    """Weights as two f16, the second scaled before it is rounded: half a step of 2^-47 of the largest weight."""
    n, Hq, H, D, L = shape
    check("f32", n, Hq, H, D, L, gap, 2.0 ** -47)
