"""Rotation by angles next to whole quarters of a turn, where a sine or a cosine is small: it keeps its relative accuracy."""
import math

import pytest
import torch

nv = pytest.importorskip("nvfp4_block_quantization_quantize_gb300")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_angles_next_to_quarters(layout):
    """What is left of a quarter is rounded twice in fp32 (2^-23 of it, of which its sine moves by as much), a sine or a cosine is
    off by at most 2^-23 of itself, and the product with 1 is exact."""
    rest = [0, 1, -1, 12345, 1 << 20, -(1 << 24) - 3, (1 << 33) + 7, -(1 << 40), (1 << 45) - 1, (1 << 52) + 12345, -(1 << 57) - 99,
            (1 << 60) + 1, -(1 << 61), (1 << 61) - 1, (1 << 61) - (1 << 36), 1 << 59]
    turns = [(q << 62) + r for q in range(4) for r in rest]
    half = len(turns)
    phases = torch.tensor([(t % (1 << 64)) - ((1 << 64) if t % (1 << 64) >> 63 else 0) for t in turns], device="cuda")
    x = torch.zeros(1, 1, 2 * half, device="cuda")
    first, second = (slice(0, half), slice(half, None)) if layout == "half" else (slice(0, None, 2), slice(1, None, 2))
    x[..., first] = 1.0                                    # (1, 0) turns to (cos, sin)
    got = nv.nvfp4_qk_norm_rope(x, x, torch.ones(1, dtype=torch.int64, device="cuda"), phases, layout=layout)
    for name in ("q", "k"):
        y = got[name][0, 0].cpu().double()
        for i, (q, r) in enumerate((q, r) for q in range(4) for r in rest):
            a = math.ldexp(2 * math.pi * r, -64)
            c, s = math.cos(a), math.sin(a)
            c, s = ((c, s), (-s, c), (-c, -s), (s, -c))[q]
            assert abs(y[first][i].item() - c) <= 2.0 ** -22 * abs(c), (q, r)
            assert abs(y[second][i].item() - s) <= 2.0 ** -22 * abs(s), (q, r)
