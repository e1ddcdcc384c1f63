"""The attention writes its outputs and as much of a workspace as it asked for, and not a byte around them."""
import ctypes

import pytest
import torch

from test_gpu_cache import Paged, gen, normal

nv = pytest.importorskip("nvfp4_block_quantization_quantize_gb300")
pytestmark = pytest.mark.gpu

PAD = 1 << 16


def padded(nbytes):
    """A buffer of a pattern with PAD bytes before and behind what a call may write."""
    return torch.full((nbytes + 2 * PAD,), 0xA5, dtype=torch.uint8, device="cuda")


def kept(buf):
    return bool((buf[:PAD] == 0xA5).all() and (buf[-PAD:] == 0xA5).all())


CASES = [
    # lens, queries of each (None: one, no offsets), Hq, H, D, x
    ([5000, 1, 0, 700], None, 8, 2, 128, "bf16"),
    ([9000], None, 24, 2, 64, "bf16"),
    ([3000, 4000], None, 8, 2, 256, "bf16"),
    ([2000, 300], [5, 3], 8, 2, 256, "f32"),
    ([100] * 40, None, 8, 8, 64, "f32"),
    ([3000, 9, 5000, 0], [300, 4, 513, 0], 8, 2, 128, "bf16"),
    ([3000, 9, 5000, 0], [300, 4, 513, 0], 12, 2, 64, "bf16"),
    ([3000, 900], [300, 129], 8, 2, 256, "bf16"),
    ([30000], [65], 8, 2, 128, "bf16"),
]


@pytest.mark.parametrize("o", ["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_nothing_around_outputs_and_workspace(i, o):
    lens, counts, Hq, H, D, x = CASES[i]
    c = Paged(i, lens, H, D, 32, "none")
    n = [1] * len(lens) if counts is None else counts
    T = sum(n) + (5 if counts else 0)                      # rows behind the last sequence
    q = normal(gen(i), T, Hq, D).to({"bf16": torch.bfloat16, "f32": torch.float32}[x])
    off = None if counts is None else torch.tensor([0] + counts, device="cuda").cumsum(0)
    lib, B, W = nv.load_library(), len(lens), c.pages.shape[1]
    dt, odt, size = (nv.F32 if x == "f32" else nv.BF16), (nv.F32 if o == "f32" else nv.BF16), 4 if o == "f32" else 2
    need = lib.nvfp4_cache_attention_workspace(T, Hq, H, D, B, W, 32, dt, int(off is not None))
    ws, out, lse = padded(need), padded(T * Hq * D * size), padded(T * Hq * 4)
    cache, pages = c.cache.clone(), c.pages.clone()
    at = lambda t, k=0: ctypes.c_void_p(0 if t is None else t.data_ptr() + k)      # noqa: E731
    rc = lib.nvfp4_cache_attention(at(q), T, Hq, Hq * D, dt, at(c.cache), c.cache.shape[0], 32, H, D, at(c.pages), B, W, at(c.lengths),
                                   at(off), nv.GAMAX_NONE, None, nv.GAMAX_NONE, None, 448.0, D ** -0.5, 1, 0, None, at(out, PAD), odt,
                                   at(lse, PAD), at(ws, PAD), need, torch.cuda.current_stream().cuda_stream)
    assert rc == nv.OK
    torch.cuda.synchronize()
    assert kept(ws) and kept(out) and kept(lse)
    assert torch.equal(c.cache, cache) and torch.equal(c.pages, pages)
    rows = out[PAD:PAD + T * Hq * D * size].view(T, -1)
    assert (rows[sum(n):] == 0xA5).all() and (lse[PAD:PAD + T * Hq * 4].view(T, -1)[sum(n):] == 0xA5).all()
    got = rows[:sum(n)].clone().view(torch.float32 if o == "f32" else torch.bfloat16).view(-1, Hq, D)
    c.check(q, n, got, lse[PAD:PAD + T * Hq * 4].view(torch.float32).view(T, Hq)[:sum(n)])
