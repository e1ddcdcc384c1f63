"""Attention whose first key takes nearly all weight and has no value, so that the output is made of small weights alone:
they keep their bits, however the kernels hold them on their way into the second product."""
import pytest
import torch

from cache_helpers import attention, parts, take, tolerance, values

nv = pytest.importorskip("nvfp4_block_quantization_quantize_gb300")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def check(x, n, Hq, H, D, L, gap, floor, near=None, share=0.0):
    """n queries on L keys, the first of which stands `gap` above the others' logits; no mask.  `floor`: half a step of the
    smallest weights, in parts of the largest: what a kernel may leave out of each of `near` keys (None: all); `share`: and of
    the sum of the others' weights."""
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
    others = torch.exp(attention(q, kk[1:], vv[1:], n, scale=1.0, causal=False)[1] - want).unsqueeze(2)
    biggest = vv.abs().max().item()
    tol = tolerance(out, mass, most, 0.0, L, D, q.dtype, got.dtype) + ((near or L) * floor + share * others) * biggest
    assert (tol < 0.5 * out).double().mean() > 0.7         # (a kernel that drops these weights fails)
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


@pytest.mark.parametrize("gap", [9.0, 15.0, 18.0])
@pytest.mark.parametrize("shape", [(300, 2, 1, 128, 4000), (70, 8, 2, 64, 6000), (520, 4, 4, 128, 3333)])
def test_many_bf16_queries(shape, gap):
    """The tensor-memory kernel: half a step of 2^-25 is 2^-29 of the largest weight in its block of 128 keys, and 2^-9 of any other
    block's sum."""
    n, Hq, H, D, L = shape
    check("bf16", n, Hq, H, D, L, gap, 2.0 ** -29, near=128, share=2.0 ** -9)


def test_many_bf16_queries_up_and_down():
    """Blocks whose logits rise and fall by some 20 nats from one to the next, with windows and causal masks among them: the
    reference follows, and sums do not leave fp32."""
    g = torch.Generator(device="cuda").manual_seed(3)
    n, Hq, H, D, L, P = 150, 4, 2, 128, 3000, 16
    level = torch.tensor([0.0, 3.0, -4.0, 6.0, -6.0, 1.0, 6.0, -6.0, -6.0, 2.0], device="cuda")
    k, v = torch.randn(L, H, D, generator=g, device="cuda"), torch.randn(L, H, D, generator=g, device="cuda")
    k[..., 0] = level[torch.arange(L, device="cuda") // 128 % 10][:, None]
    j = torch.arange(L, device="cuda")
    cache = nv.nvfp4_cache_empty(-(-L // P), P, H, D)
    nv.nvfp4_cache_write(cache, k, v, j)
    q = torch.randn(n, Hq, D, generator=g, device="cuda")
    q[..., 0] = torch.tensor([40.0, -40.0, 100.0, 400.0], device="cuda")
    q = q.to(torch.bfloat16)
    kc, ks, vc, vs = (take(p, j) for p in parts(cache))
    kk, vv = values(kc, ks), values(vc, vs)
    for opt in ({}, {"window": 700}, {"causal": False}):
        got, lse = nv.nvfp4_cache_attention(q, cache, j[:cache.shape[0]].int().view(1, -1), torch.tensor([L], device="cuda"), want_lse=True,
                                            offsets=torch.tensor([0, n], device="cuda"), out_dtype="f32", **opt)
        out, want, mass, most = attention(q, kk, vv, n, scale=D ** -0.5, **opt)
        tol = tolerance(out, mass, most, vv.abs().max().item(), L, D, q.dtype, got.dtype)
        assert ((got.double() - out).abs() <= tol).all()
        assert ((lse.double() - want).abs() <= (D + 8) * 2.0 ** -23 * most + 2.0 ** -22 * want.abs() + (L / 16 + 64) * 2.0 ** -23).all()
