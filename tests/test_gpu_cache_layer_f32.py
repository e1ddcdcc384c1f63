"""FP4Attention on fp32 inputs: nothing between its two products is held in fewer bits."""
import pytest
import torch

from cache_helpers import attention, parts, take, tolerance, values

nv = pytest.importorskip("nvfp4_block_quantization_quantize_gb300")
serving = pytest.importorskip("nvfp4_block_quantization_quantize_gb300.serving")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("M", [1, 16, 40])
def test_a_layer_in_fp32(M, norm):
    """The layer is its operators in fp32, and their queries and attention are as exact as fp32 ones."""
    g = torch.Generator(device="cuda").manual_seed(M)

    def normal(*s):
        return torch.randn(*s, generator=g, device="cuda")

    w = [1 + 0.1 * normal(64) if norm else None for _ in range(2)]
    phases = nv.nvfp4_rope_phases(64, device="cuda")
    lay = serving.FP4Attention(1 + 0.1 * normal(512), normal(12 * 64, 512) * 512 ** -0.5, normal(512, 512) * 512 ** -0.5, 8, 2,
                               phases=phases, q_norm=w[0], k_norm=w[1], window=30, sinks=normal(8))
    x, hid = normal(M, 512), normal(M, 512)
    a, b = (nv.nvfp4_cache_empty(4, 16, 2, 64) for _ in range(2))
    pages, j = torch.tensor([[2, 0, 3, 1]], dtype=torch.int32, device="cuda"), torch.arange(M, device="cuda")
    slots = pages[0].long()[j // 16] * 16 + j % 16
    ln, off = torch.tensor([M], device="cuda"), torch.tensor([0, M], device="cuda")
    got, hidden = lay(x, hid, a, pages, ln, slots, j, off)
    assert got.dtype == hidden.dtype == torch.float32

    y, h = lay.qkv(x, hid, "f32")
    y = y.view(M, 12, 64)
    q = nv.nvfp4_qk_norm_rope(y[:, :8], y[:, 8:10], j, phases, q_weight=w[0], k_weight=w[1], cache=b, v=y[:, 10:], slots=slots)["q"]
    o = nv.nvfp4_cache_attention(q, b, pages, ln, offsets=off, window=30, sinks=lay.sinks, out_dtype="f32")
    assert y.dtype == q.dtype == o.dtype == torch.float32
    assert torch.equal(hidden, h) and torch.equal(a, b)
    assert torch.equal(got, lay.back.product(o.view(M, 512), "f32"))
    kc, ks, vc, vs = (take(p, slots) for p in parts(b))
    k, v = values(kc, ks), values(vc, vs)
    out, _, mass, most = attention(q, k, v, M, scale=64 ** -0.5, window=30, sinks=lay.sinks)
    assert ((o.double() - out).abs() <= tolerance(out, mass, most, v.abs().max().item(), M, 64, q.dtype, o.dtype)).all()
