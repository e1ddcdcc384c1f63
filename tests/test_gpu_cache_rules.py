"""Where the work of a few sequences is cut between CTAs: the workspace's size tells."""
import pytest

nv = pytest.importorskip("nvfp4_block_quantization_quantize_gb300")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,dtype,keys", [(128, nv.BF16, 1216), (64, nv.F32, 1216), (256, nv.BF16, 1040), (128, nv.F32, 1040),
                                          (256, nv.F32, 784)])
def test_few_groups_are_cut_by_what_a_tile_takes(D, dtype, keys):
    """The keys from which one group's work is cut (and needs a workspace): fewer where a tile takes longer."""
    ws = nv.load_library().nvfp4_cache_attention_workspace
    assert ws(1, 4, 1, D, 1, keys // 16 - 1, 16, dtype, 0) == 0 < ws(1, 4, 1, D, 1, keys // 16, 16, dtype, 0)


@pytest.mark.parametrize("D,dtype", [(128, nv.BF16), (64, nv.F32), (256, nv.BF16), (128, nv.F32), (256, nv.F32)])
def test_many_groups_are_not_cut_earlier(D, dtype):
    ws = nv.load_library().nvfp4_cache_attention_workspace
    assert ws(16, 64, 8, D, 16, 1200 // 16, 16, dtype, 0) == 0 < ws(16, 64, 8, D, 16, 1216 // 16, 16, dtype, 0)
