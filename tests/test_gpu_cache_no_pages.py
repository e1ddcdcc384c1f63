"""A cache without a page: every slot lies outside it."""
import pytest
import torch

nv = pytest.importorskip("nvfp4_block_quantization_quantize_gb300")
pytestmark = pytest.mark.gpu


def test_calls_on_a_cache_without_pages():
    q, k = (torch.randn(5, h, 64, device="cuda").to(torch.bfloat16) for h in (4, 2))
    slots = torch.tensor([0, -1, 7, 1 << 40, 3], device="cuda")
    pos, ph = torch.arange(5, device="cuda"), nv.nvfp4_rope_phases(64, device="cuda")
    cache = nv.nvfp4_cache_empty(0, 16, 2, 64)
    nv.nvfp4_cache_write(cache, k, k, slots)
    assert all((t == 0).all() for t in nv.nvfp4_cache_read(cache, slots))
    r = nv.nvfp4_qk_norm_rope(q, k, pos, ph, cache=cache, v=k, slots=slots)
    assert set(r) == {"q"} and torch.equal(r["q"], nv.nvfp4_qk_norm_rope(q, k, pos, ph)["q"])
    o = nv.nvfp4_cache_attention(q, cache, torch.zeros(5, 2, dtype=torch.int32, device="cuda"), torch.full((5,), 9, device="cuda"))
    assert (o == 0).all()
