"""The README's examples run as they stand, given the names that their comments describe."""
import os
import re

import pytest
import torch

nv = pytest.importorskip("nvfp4_block_quantization_quantize_gb300")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def blocks():
    with open(os.path.join(ROOT, "README.md")) as f:
        return re.findall(r"```python\n(.*?)```", f.read(), re.S)


def names(first):
    """What an example that begins with `first` takes as given."""
    def normal(*shape):
        return torch.randn(*shape, device="cuda").to(torch.bfloat16)

    if first == "import torch":
        return {}
    if first.startswith("n = nv.nvfp4_rmsnorm"):
        w = [nv.nvfp4_quantize(normal(256, 128)) for _ in range(3)]
        return dict(x=normal(9, 128), norm_weight=torch.ones(128, device="cuda"), hidden=normal(9, 128), q=w[0],
                    w_codes=torch.stack([t["codes"] for t in w]), w_scales=torch.stack([t["scales"] for t in w]),
                    w_amax=torch.ones(3, device="cuda"), rows=torch.arange(9, device="cuda"),
                    offsets=torch.tensor([0, 2, 2, 9], device="cuda"))
    assert first.startswith("phases = nv.nvfp4_rope_phases")
    T = 70
    return dict(qkv=normal(T, 48, 128), positions=torch.arange(T, device="cuda"), wq=torch.ones(128, device="cuda"),
                wk=torch.ones(128, device="cuda"), slots=torch.arange(T, device="cuda"),
                page_table=torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), lengths=torch.tensor([T], device="cuda"),
                offsets=torch.tensor([0, T], device="cuda"))


@pytest.mark.parametrize("i", range(len(blocks())))
def test_readme_example(i):
    src = blocks()[i]
    scope = {"nv": nv, "torch": torch, **names(src.splitlines()[0])}
    exec(compile(src, f"README block {i}", "exec"), scope)
    torch.cuda.synchronize()
    if "phases" in scope:
        assert scope["o"].shape == (70, 32, 128) and scope["o"].isfinite().all() and scope["k"].shape == (70, 8, 128)
