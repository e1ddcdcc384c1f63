"""How the cache operators are called: the binding's short path against the Python one, other streams, captured and
replayed calls, sizes at the ends, pages and lengths that are wrong, caches past 2^32 bytes, and the layer made of
them over several steps."""
import ctypes
import math

import pytest
import torch

from cache_helpers import attention, parts, take, tolerance, values
from test_gpu_cache import Paged, gen, normal

nv = pytest.importorskip("nvfp4_block_quantization_quantize_gb300")
serving = pytest.importorskip("nvfp4_block_quantization_quantize_gb300.serving")
pytestmark = pytest.mark.gpu


def small(seed=1, x=torch.bfloat16, n=1, lens=(37, 700, 5), Hq=8, H=2, D=128, P=16):
    c = Paged(seed, list(lens), H, D, P, "head")
    q = (2 * normal(gen(seed + 50), n * len(lens), Hq, D)).to(x)
    return c, q, dict(k_gamax=c.ka, v_gamax=c.va)


# ---- both ways into a call ------------------------------------------------------------------------
def test_both_paths_of_the_binding_give_the_same(monkeypatch):
    c, q, kw = small()
    g = gen(9)
    qkv = normal(g, 3, 12, 128).to(torch.bfloat16)
    pos, ph = torch.tensor([4, 9, 1 << 33], device="cuda"), nv.nvfp4_rope_phases(128, device="cuda")
    w = normal(g, 128)
    slots = torch.tensor([3, -1, 40], device="cuda")
    off = torch.tensor([0, 1, 2, 3], device="cuda")

    def all_calls():
        cache = c.cache.clone()
        r = nv.nvfp4_qk_norm_rope(qkv[:, :8], qkv[:, 8:10], pos, ph, q_weight=w, k_weight=w, layout="interleaved")
        f = nv.nvfp4_qk_norm_rope(qkv[:, :8], qkv[:, 8:10], pos, ph, cache=cache, v=qkv[:, 10:], slots=slots, **kw)
        n = nv.nvfp4_qk_norm_rope(qkv[:, :8], qkv[:, 8:10], None, None, q_weight=w, k_weight=w)
        nv.nvfp4_cache_write(cache, qkv[:, 8:10], qkv[:, 10:], slots + 5, **kw)
        k, v = nv.nvfp4_cache_read(cache, slots + 5, out_dtype="f32", **kw)
        o, lse = nv.nvfp4_cache_attention(q, c.cache, c.pages, c.lengths, want_lse=True, window=9, **kw)
        s = nv.nvfp4_cache_attention(q, c.cache, c.pages, c.lengths, offsets=off, scale=0.2, sinks=w[:8], out_dtype="f32",
                                     causal=False, **kw)
        return [r["q"], r["k"], f["q"], n["q"], n["k"], cache, k, v, o, lse, s]

    short = all_calls()
    monkeypatch.setattr(nv, "_call", nv._NoShortPath)
    for a, b in zip(short, all_calls()):
        assert a.shape == b.shape and a.dtype == b.dtype and torch.equal(a, b)


def test_the_short_path_is_taken_and_leaves_other_calls():
    c, q, kw = small()
    args = [q, c.cache, c.pages, c.lengths, None, c.ka, c.va, 448.0, None, True, 0, None, "bf16", None, False]
    assert torch.is_tensor(nv._call.cache_attention(*args))
    assert nv._call.cache_attention(*(args[:9] + [1] + args[10:])) is None          # causal is not a bool
    assert nv._call.cache_attention(*([q.cpu()] + args[1:])) is None
    assert nv._call.cache_attention(*([q.transpose(0, 1)] + args[1:])) is None
    assert nv._call.cache_attention(*(args[:3] + [c.lengths.int()] + args[4:])) is None
    assert nv._call.cache_write(c.cache, q[:, :2], q[:, 2:4], torch.tensor([1, 2, 3], device="cuda"), None, None, 448.0) is True


def test_given_outputs_are_returned_and_written():
    c, q, kw = small()
    o = torch.empty(3, 8, 128, device="cuda", dtype=torch.bfloat16)
    assert nv.nvfp4_cache_attention(q, c.cache, c.pages, c.lengths, out=o, **kw) is o
    assert torch.equal(o, nv.nvfp4_cache_attention(q, c.cache, c.pages, c.lengths, **kw))
    k = q[:, :2].contiguous()
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    r = nv.nvfp4_qk_norm_rope(q, k, None, None, q_out=qo, k_out=ko)
    assert r["q"] is qo and r["k"] is ko and torch.equal(qo, q) and torch.equal(ko, k)


def test_binding_refuses_what_does_not_fit():
    c, q, kw = small()
    i3 = torch.arange(3, device="cuda")
    k = q[:, :2]
    for call in (lambda: nv.nvfp4_cache_attention(q, c.cache, c.pages.long(), c.lengths),
                 lambda: nv.nvfp4_cache_attention(q, c.cache, c.pages, c.lengths[:2]),
                 lambda: nv.nvfp4_cache_attention(q[..., :64], c.cache, c.pages, c.lengths),
                 lambda: nv.nvfp4_cache_attention(q, c.cache.cpu(), c.pages, c.lengths),
                 lambda: nv.nvfp4_cache_attention(q, c.cache, c.pages, c.lengths, sinks=torch.zeros(7, device="cuda")),
                 lambda: nv.nvfp4_cache_attention(q, c.cache, c.pages, c.lengths, k_gamax=torch.ones(3, device="cuda")),
                 lambda: nv.nvfp4_cache_attention(q, c.cache, c.pages, c.lengths, out=torch.empty(3, 8, 128, device="cuda")),
                 lambda: nv.nvfp4_cache_attention(q, c.cache, c.pages, c.lengths, out_dtype="f16"),
                 lambda: nv.nvfp4_cache_write(c.cache, k, k.float(), i3),
                 lambda: nv.nvfp4_cache_write(c.cache, q, q, i3),
                 lambda: nv.nvfp4_cache_write(c.cache, k, k, i3[:2]),
                 lambda: nv.nvfp4_cache_write(c.cache.transpose(0, 1), k, k, i3),
                 lambda: nv.nvfp4_cache_read(c.cache, i3.int()),
                 lambda: nv.nvfp4_cache_read(c.cache[..., :1000], i3),
                 lambda: nv.nvfp4_qk_norm_rope(q, k, i3, None),
                 lambda: nv.nvfp4_qk_norm_rope(q, k, None, None, q_weight=torch.ones(128, device="cuda")),
                 lambda: nv.nvfp4_qk_norm_rope(q, k, None, None, cache=c.cache),
                 lambda: nv.nvfp4_qk_norm_rope(q, k, None, None, k_gamax=c.ka),
                 lambda: nv.nvfp4_qk_norm_rope(q, k, None, None, layout="third"),
                 lambda: nv.nvfp4_qk_norm_rope(q, k[:2], None, None)):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_cache_attention(q, c.cache, c.pages, c.lengths, scale=math.nan)
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_cache_attention(q[:, :7], c.cache, c.pages, c.lengths)
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_cache_attention(q, c.cache, c.pages, c.lengths, window=-4)


# ---- streams and graphs ---------------------------------------------------------------------------
def test_calls_run_on_the_given_stream():
    c, q, kw = small()
    want = nv.nvfp4_cache_attention(q, c.cache, c.pages, c.lengths, **kw)
    side = torch.cuda.Stream()
    slots = torch.arange(3, device="cuda")
    cache = torch.zeros_like(c.cache)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)                      # what follows on the side stream comes late
        c2 = c.cache.clone()
    got = nv.nvfp4_cache_attention(q, c2, c.pages, c.lengths, stream=side, **kw)
    nv.nvfp4_cache_write(cache, q[:, :2], q[:, 2:4], slots, stream=side.cuda_stream)
    k, v = nv.nvfp4_cache_read(cache, slots, stream=side, out_dtype="f32")
    r = nv.nvfp4_qk_norm_rope(q, q[:, :2], None, None, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(r["q"], q)
    plain = torch.zeros_like(c.cache)
    nv.nvfp4_cache_write(plain, q[:, :2], q[:, 2:4], slots)
    assert torch.equal(cache, plain) and torch.equal(k, nv.nvfp4_cache_read(plain, slots, out_dtype="f32")[0])


def test_two_calls_at_once():
    """Each has a workspace of its own."""
    jobs = [small(s, lens=(9000, 12, 3000)) for s in (1, 2, 3, 4)]
    want = [nv.nvfp4_cache_attention(q, c.cache, c.pages, c.lengths, **kw) for c, q, kw in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for (c, q, kw), s in zip(jobs, streams):
            with torch.cuda.stream(s):
                got.append(nv.nvfp4_cache_attention(q, c.cache, c.pages, c.lengths, **kw))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("Hq", [8, 96])                    # a few rows a sequence, and many (the tensor-memory kernel)
def test_a_captured_call_follows_its_inputs(Hq):
    """Lengths, offsets, tables and contents are read on the device: a graph serves whatever they hold."""
    c, q, kw = small(3, lens=(3000, 900, 60), n=3, Hq=Hq)
    lengths, offsets, pages = c.lengths.clone(), torch.tensor([0, 3, 6, 9], device="cuda"), c.pages.clone()
    out = torch.empty(9, Hq, 128, device="cuda", dtype=torch.bfloat16)
    call = lambda: nv.nvfp4_cache_attention(q, c.cache, pages, lengths, offsets=offsets, out=out, **kw)      # noqa: E731
    call()
    torch.cuda.synchronize()
    a, b = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(a):
        call()
    with torch.cuda.graph(b, pool=a.pool()):               # shares its memory, the workspace's too
        call()
    for lens, off in (([3000, 900, 60], [0, 3, 6, 9]), ([1, 0, 60], [0, 1, 1, 9]), ([2999, 17, 33], [0, 0, 8, 9]),
                      ([0, 0, 0], [0, 0, 0, 0]), ([2000, 900, 1], [0, 8, 9, 9])):
        lengths.copy_(torch.tensor(lens))
        offsets.copy_(torch.tensor(off))
        out.fill_(7.0)
        a.replay()
        b.replay()
        got = out.clone()
        out.fill_(7.0)
        call()
        assert torch.equal(got, out)
        assert (out[off[-1]:] == 7).all()                  # rows behind the last sequence stay as they were
        c.lens = lens
        c.check(q, [y - x for x, y in zip(off, off[1:])], got)


# ---- ends -----------------------------------------------------------------------------------------
def test_empty_batches():
    cache = nv.nvfp4_cache_empty(4, 16, 2, 64)
    e = torch.empty(0, 4, 64, device="cuda", dtype=torch.bfloat16)
    i = torch.empty(0, dtype=torch.int64, device="cuda")
    assert nv.nvfp4_cache_attention(e, cache, torch.empty(0, 3, dtype=torch.int32, device="cuda"), i).shape == (0, 4, 64)
    assert nv.nvfp4_cache_read(cache, i)[0].shape == (0, 2, 64)
    nv.nvfp4_cache_write(cache, e[:, :2], e[:, :2], i)
    assert nv.nvfp4_qk_norm_rope(e, e[:, :2], i, nv.nvfp4_rope_phases(64, device="cuda"))["q"].shape == (0, 4, 64)
    q = normal(gen(1), 2, 4, 64)
    o, lse = nv.nvfp4_cache_attention(q, cache, torch.empty(2, 0, dtype=torch.int32, device="cuda"),
                                      torch.tensor([5, 0], device="cuda"), want_lse=True)      # no pages: no keys
    assert (o == 0).all() and torch.isneginf(lse).all()


def test_wrong_lengths_offsets_and_pages():
    """Lengths are clamped to the table, offsets to the batch; keys of pages that do not exist are not seen."""
    c, q, kw = small(5, lens=(64, 40, 48), P=16)
    want = nv.nvfp4_cache_attention(q, c.cache, c.pages, c.lengths, **kw)
    long = torch.tensor([1 << 40, 40, 48], device="cuda")
    assert torch.equal(nv.nvfp4_cache_attention(q, c.cache, c.pages, long, **kw), want)      # 4 pages of 16: 64
    got = nv.nvfp4_cache_attention(q, c.cache, c.pages, torch.tensor([64, -5, 48], device="cuda"), **kw)
    assert torch.equal(got[[0, 2]], want[[0, 2]]) and (got[1] == 0).all()
    off = torch.tensor([-9, 1, 2, 1 << 50], device="cuda")
    assert torch.equal(nv.nvfp4_cache_attention(q, c.cache, c.pages, c.lengths, offsets=off, **kw), want)
    for bad in (-1, c.cache.shape[0], 1 << 30, -(1 << 31)):
        pages = c.pages.clone()
        pages[0, 1] = bad
        got = nv.nvfp4_cache_attention(q, c.cache, pages, c.lengths, out_dtype="f32", **kw)
        k, v = c.values(0)
        keep = torch.ones(64, dtype=torch.bool, device="cuda")
        keep[16:32] = False
        out, _, mass, most = attention(q[:1], k[keep], v[keep], 1, scale=128 ** -0.5, causal=False)
        assert ((got[:1].double() - out).abs() <= tolerance(out, mass, most, v.abs().max().item(), 64, 128, q.dtype, got.dtype)).all()


@pytest.mark.parametrize("L", [300, 2000])                # the second by the tensor-memory kernel
def test_many_rows_of_wrong_pages(L):
    c, q, kw = small(6, lens=(L, 200), n=1, P=16, H=1, Hq=1)
    q = (2 * normal(gen(3), 300, 1, 128)).to(torch.bfloat16)
    off = torch.tensor([0, 150, 300], device="cuda")
    pages = c.pages.clone()
    pages[0, 5] = -1
    got = nv.nvfp4_cache_attention(q, c.cache, pages, c.lengths, offsets=off, causal=False, out_dtype="f32", **kw)
    k, v = c.values(0)
    keep = torch.ones(L, dtype=torch.bool, device="cuda")
    keep[80:96] = False
    out, _, mass, most = attention(q[:150], k[keep], v[keep], 150, scale=128 ** -0.5, causal=False)
    assert ((got[:150].double() - out).abs() <= tolerance(out, mass, most, v.abs().max().item(), L, 128, q.dtype, got.dtype)).all()


@pytest.mark.parametrize("n,L", [(1, 50), (100, 50), (100, 1500)])
def test_a_shared_page_and_infinities_stay_in_their_rows(n, L):
    c, q, kw = small(7, lens=(L, L), n=1, Hq=2, H=1)
    q = (2 * normal(gen(4), 2 * n, 2, 128)).to(torch.bfloat16)
    off = None if n == 1 else torch.tensor([0, n, 2 * n], device="cuda")
    pages = c.pages.clone()
    pages[1] = pages[0]                                    # both sequences are the same keys
    q[n:] = q[:n]
    a = nv.nvfp4_cache_attention(q, c.cache, pages, c.lengths, offsets=off, **kw)
    if L == 50:                                            # (longer groups may be cut between CTAs, each elsewhere)
        assert torch.equal(a[:n], a[n:])
    k, v = c.values(0)
    out, _, mass, most = attention(q[:n], k, v, n, scale=128 ** -0.5)
    tol = tolerance(out, mass, most, v.abs().max().item(), L, 128, q.dtype, a.dtype)
    assert ((a[:n].double() - out).abs() <= tol).all() and ((a[n:].double() - out).abs() <= tol).all()
    q[0, 0, 3], q[n, 1, 5] = math.inf, math.nan
    b = nv.nvfp4_cache_attention(q, c.cache, pages, c.lengths, offsets=off, causal=False, **kw)
    q[0, 0, 3], q[n, 1, 5] = 0.0, 0.0
    want = nv.nvfp4_cache_attention(q, c.cache, pages, c.lengths, offsets=off, causal=False, **kw)
    bad = torch.zeros(2 * n, 2, dtype=torch.bool, device="cuda")
    bad[0, 0] = bad[n, 1] = True
    assert torch.equal(b[~bad], want[~bad]) and b[bad].isnan().all()


@pytest.mark.parametrize("scale", [1e-3, 30.0, 3000.0])
def test_large_and_small_queries(scale):
    """Logits far apart: one key takes all weight, in both kernels; f16 holds the queries by their power of two."""
    for n, Hq in ((1, 4), (70, 4)):
        c = Paged(8, [2000, 300], 2, 128, 16, "none")
        q = (scale * normal(gen(5), 2 * n, Hq, 128)).to(torch.bfloat16)
        off = torch.tensor([0, n, 2 * n], device="cuda")
        got, lse = nv.nvfp4_cache_attention(q, c.cache, c.pages, c.lengths, offsets=off, out_dtype="f32", want_lse=True)
        c.check(q, [n, n], got, lse)


@pytest.mark.parametrize("n", [1, 300])
def test_one_page_past_32_bits(n):
    """A page of over 2^31 bytes, its last tokens used, by a few rows and by many."""
    D, L = 128, 1100
    P = ((1 << 31) // (18 * D) + 200) * 16
    cache = torch.empty(2, 1, P // 16, 18 * D, dtype=torch.uint8, device="cuda")
    g = gen(5)
    k, v = normal(g, L, 1, D), normal(g, L, 1, D)
    slots = 2 * P - L + torch.arange(L, device="cuda")
    nv.nvfp4_cache_write(cache, k, v, slots)
    tiny = nv.nvfp4_cache_empty(1, 1104, 1, D)
    nv.nvfp4_cache_write(tiny, k, v, torch.arange(L, device="cuda") + 4)      # (as far into a tile: P - L is 4 more than tiles)
    for x, y in zip(nv.nvfp4_cache_read(cache, slots), nv.nvfp4_cache_read(tiny, torch.arange(L, device="cuda") + 4)):
        assert torch.equal(x, y)
    q = normal(g, n, 4, D).to(torch.bfloat16)
    kw = dict(offsets=torch.tensor([0, n], device="cuda"), window=L - n, out_dtype="f32")
    got = nv.nvfp4_cache_attention(q, cache, torch.tensor([[1]], dtype=torch.int32, device="cuda"), torch.tensor([P], device="cuda"), **kw)
    kc, ks, vc, vs = (take(x, torch.arange(L, device="cuda") + 4) for x in parts(tiny))
    k, v = values(kc, ks, None), values(vc, vs, None)
    out, _, mass, most = attention(q, k, v, n, scale=D ** -0.5, window=L - n)
    assert ((got.double() - out).abs() <= tolerance(out, mass, most, v.abs().max().item(), L, D, q.dtype, got.dtype)).all()


def test_slots_past_32_bits():
    """A cache of over 2^32 bytes, its last pages used."""
    D, H, P = 256, 8, 128
    pages = (1 << 32) // (H * P // 16 * 18 * D) + 40
    cache = torch.empty(pages, H, P // 16, 18 * D, dtype=torch.uint8, device="cuda")
    assert cache.numel() > 1 << 32
    g = gen(2)
    table = torch.tensor([[pages - 1, 3, pages - 20]], dtype=torch.int32, device="cuda")
    L = 300
    j = torch.arange(L, device="cuda")
    slots = table[0].long()[j // P] * P + j % P
    k, v = normal(g, L, H, D), normal(g, L, H, D)
    nv.nvfp4_cache_write(cache, k, v, slots)
    tiny = nv.nvfp4_cache_empty(3, P, H, D)
    nv.nvfp4_cache_write(tiny, k, v, j)
    for a, b in zip(nv.nvfp4_cache_read(cache, slots), nv.nvfp4_cache_read(tiny, j)):
        assert torch.equal(a, b)
    q = normal(g, 1, 16, D).to(torch.bfloat16)
    ln = torch.tensor([L], device="cuda")
    want = nv.nvfp4_cache_attention(q, tiny, torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda"), ln)
    assert torch.equal(nv.nvfp4_cache_attention(q, cache, table, ln), want)


def test_many_queries_in_a_cache_past_32_bits():
    D, H, P = 128, 8, 128
    pages = (1 << 32) // (H * P // 16 * 18 * D) + 9
    cache = torch.empty(pages, H, P // 16, 18 * D, dtype=torch.uint8, device="cuda")
    g = gen(3)
    table = torch.tensor([[pages - 1, pages - 7]], dtype=torch.int32, device="cuda")
    j = torch.arange(256, device="cuda")
    k, v = normal(g, 256, H, D), normal(g, 256, H, D)
    nv.nvfp4_cache_write(cache, k, v, table[0].long()[j // P] * P + j % P)
    tiny = nv.nvfp4_cache_empty(2, P, H, D)
    nv.nvfp4_cache_write(tiny, k, v, j)
    q, ln, off = normal(g, 130, 64, D).to(torch.bfloat16), torch.tensor([256], device="cuda"), torch.tensor([0, 130], device="cuda")
    want = nv.nvfp4_cache_attention(q, tiny, torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), ln, offsets=off)
    assert torch.equal(nv.nvfp4_cache_attention(q, cache, table, ln, offsets=off), want)


def test_outputs_at_16_bytes():
    """Addresses on 16 bytes and not on 32, for outputs and workspace (the C call)."""
    c, q, kw = small(11, lens=(5000, 700, 900), n=30, Hq=8)
    off = torch.tensor([0, 30, 60, 90], device="cuda")
    want, lse = nv.nvfp4_cache_attention(q, c.cache, c.pages, c.lengths, offsets=off, want_lse=True, **kw)
    lib = nv.load_library()
    for T, o in ((90, off), (3, None)):
        B, W, dt = 3, c.pages.shape[1], nv.BF16
        need = lib.nvfp4_cache_attention_workspace(T, 8, 2, 128, B, W, 16, dt, int(o is not None))
        ws = torch.empty(need + 64, dtype=torch.uint8, device="cuda")
        out = torch.empty(T * 8 * 128 + 64, dtype=torch.bfloat16, device="cuda")
        at = lambda t, n: ctypes.c_void_p(t.data_ptr() + n)      # noqa: E731
        rc = lib.nvfp4_cache_attention(at(q, 0), T, 8, 8 * 128, dt, at(c.cache, 0), c.cache.shape[0], 16, 2, 128, at(c.pages, 0),
                                       B, W, at(c.lengths, 0), None if o is None else at(o, 0), nv.GAMAX_ROW_GIVEN,
                                       at(c.ka, 0), nv.GAMAX_ROW_GIVEN, at(c.va, 0), 448.0, 128 ** -0.5, 1, 0, None,
                                       at(out, 16), dt, None, at(ws, 16), need, torch.cuda.current_stream().cuda_stream)
        assert rc == nv.OK
        got = out[8:8 + T * 8 * 128].view(T, 8, 128)
        assert torch.equal(got, want if o is not None else nv.nvfp4_cache_attention(q[:3], c.cache, c.pages, c.lengths, **kw))


# ---- the layer ------------------------------------------------------------------------------------
def layer(g, D_model=512, Hq=8, H=2, D=64, **kw):
    mk = lambda *s: (normal(g, *s) * s[-1] ** -0.5).to(torch.bfloat16)      # noqa: E731
    return serving.FP4Attention((1 + 0.1 * normal(g, D_model)).to(torch.bfloat16), mk((Hq + 2 * H) * D, D_model),
                                mk(D_model, Hq * D), Hq, H, phases=nv.nvfp4_rope_phases(D, device="cuda"),
                                q_norm=1 + 0.1 * normal(g, D), k_norm=1 + 0.1 * normal(g, D), **kw)


def test_a_layer_over_a_prompt_and_steps():
    """Two sequences: their prompts at once, then tokens one at a time in a captured step; what the attention gave is
    checked against the cache's own values, and the whole against the same operators called one by one."""
    g = gen(21)
    lay = layer(g, k_gamax=torch.full((2,), 20.0, device="cuda"), v_gamax=torch.full((1,), 8.0, device="cuda"), window=40)
    P, W = 16, 6
    cache = nv.nvfp4_cache_empty(2 * W, P, 2, 64)
    pages = torch.randperm(2 * W, generator=g, device="cuda").int().view(2, W)
    prompts = [33, 50]

    def place(b, j):
        return pages[b].long()[j // P] * P + j % P

    def direct(x, hidden, lengths, slots, positions, offsets):
        y, hidden = lay.qkv(x, hidden, "bf16")
        y = y.view(x.shape[0], 12, 64)
        q = nv.nvfp4_qk_norm_rope(y[:, :8], y[:, 8:10], positions, lay.rope["phases"], q_weight=lay.rope["q_weight"],
                                  k_weight=lay.rope["k_weight"], eps=lay.rope["eps"], cache=cache, v=y[:, 10:], slots=slots, **lay.gamax)["q"]
        o, lse = nv.nvfp4_cache_attention(q, cache, pages, lengths, offsets=offsets, window=40, want_lse=True, **lay.gamax)
        return q, o, lay.back.product(o.view(x.shape[0], 512), "bf16"), hidden

    def checked(q, o, lens, counts):
        row = 0
        for b, n in enumerate(counts):
            kc, ks, vc, vs = (take(p, place(b, torch.arange(lens[b], device="cuda"))) for p in parts(cache))
            k, v = values(kc, ks, lay.gamax["k_gamax"]), values(vc, vs, lay.gamax["v_gamax"])
            out, _, mass, most = attention(q[row:row + n], k, v, n, scale=64 ** -0.5, window=40)
            assert ((o[row:row + n].double() - out).abs() <= tolerance(out, mass, most, v.abs().max().item(), lens[b], 64, q.dtype, o.dtype)).all()
            row += n

    M = sum(prompts)
    x, hid = normal(g, M, 512).to(torch.bfloat16), normal(g, M, 512).to(torch.bfloat16)
    pos = torch.cat([torch.arange(n, device="cuda") for n in prompts])
    slots = torch.cat([place(b, torch.arange(n, device="cuda")) for b, n in enumerate(prompts)])
    off, lengths = torch.tensor([0, 33, 83], device="cuda"), torch.tensor(prompts, device="cuda")
    got = lay(x, hid, cache, pages, lengths, slots, pos, off)
    after = cache.clone()
    q, o, y, h = direct(x, hid, lengths, slots, pos, off)
    assert torch.equal(got[0], y) and torch.equal(got[1], h) and torch.equal(cache, after) and y.abs().sum() > 0
    checked(q, o, prompts, prompts)

    xs, hs = x[:2].clone(), hid[:2].clone()
    sl, ps, ln = torch.zeros(2, dtype=torch.int64, device="cuda"), lengths.clone(), lengths.clone()

    def feed(step):
        ln.copy_(lengths + step + 1)
        ps.copy_(ln - 1)
        sl.copy_(torch.stack([place(b, ps[b]) for b in range(2)]))
        xs.copy_(normal(g, 2, 512).to(torch.bfloat16))
        hs.copy_(normal(g, 2, 512).to(torch.bfloat16))

    feed(0)
    lay(xs, hs, cache, pages, ln, sl, ps)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = lay(xs, hs, cache, pages, ln, sl, ps)
    for step in range(40):
        feed(step)
        graph.replay()
        out, hidden = res[0].clone(), res[1].clone()
        q, o, y, h = direct(xs, hs, ln, sl, ps, None)
        assert torch.equal(out, y) and torch.equal(hidden, h)
        checked(q, o, ln.tolist(), [1, 1])


@pytest.mark.parametrize("M", [1, 16, 17, 70])
def test_a_layer_follows_its_weights(M):
    """One sequence of M tokens from nothing, 4-bit weights and all, near the same layer in 64 bits on the unquantized
    weights: far above what an error in wiring would leave (a wrong head or position gives differences of the
    values' own size)."""
    g = gen(31)
    qkv, out, nw = normal(g, 12 * 64, 512) * 512 ** -0.5, normal(g, 512, 512) * 512 ** -0.5, 1 + 0.1 * normal(g, 512)
    lay = serving.FP4Attention(nw, qkv, out, 8, 2, phases=nv.nvfp4_rope_phases(64, device="cuda"))
    x, hid = normal(g, M, 512), normal(g, M, 512)
    cache = nv.nvfp4_cache_empty(5, 16, 2, 64)
    pages, j = torch.arange(5, device="cuda").int().view(1, 5), torch.arange(M, device="cuda")
    y, h = lay(x, hid, cache, pages, torch.tensor([M], device="cuda"), j, j, torch.tensor([0, M], device="cuda"))
    assert y.dtype == torch.float32 and torch.equal(h, x + hid)
    z = h.double()
    z = z / torch.sqrt(z.square().mean(dim=1, keepdim=True) + 1e-6) * nw.double()
    t = (z @ qkv.double().t()).view(M, 12, 64)
    from cache_helpers import rotate
    freq = torch.tensor([1e4 ** (-2 * i / 64) for i in range(32)], dtype=torch.float64, device="cuda")
    q, k = rotate(t[:, :8], j, freq, "half", 1.0), rotate(t[:, 8:10], j, freq, "half", 1.0)
    o = attention(q, k, t[:, 10:], M, scale=64 ** -0.5)[0].reshape(M, 512)
    want = o @ out.double().t()
    rel = ((y.double() - want).norm() / want.norm()).item()
    # 4-bit weights, values and (above 16 rows) activations are each off by about 0.1 in the mean square; four of them in turn,
    # and the softmax on keys as far off
    assert rel < 0.45


def test_a_layer_refuses():
    g = gen(41)
    with pytest.raises(ValueError, match="FP4Attention"):
        serving.FP4Attention(None, normal(g, 12 * 64, 512), normal(g, 512, 512), 8, 3, phases=None)
    with pytest.raises(ValueError, match="FP4Attention"):
        serving.FP4Attention(None, normal(g, 12 * 64, 512), normal(g, 256, 512), 8, 2, phases=None)
