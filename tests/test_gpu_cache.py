"""The operators of a cache of keys and values in NVFP4 on the GPU, against plain forms in 64 bits; what is
quantized, against nvfp4_quantize and nvfp4_dequantize bit for bit."""
import math

import pytest
import torch

from cache_helpers import attention, parts, rotate, take, tolerance, values

nv = pytest.importorskip("nvfp4_block_quantization_quantize_gb300")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def amaxes(mode, H, g):
    if mode == "none":
        return None
    return 4.0 + torch.rand(1 if mode == "tensor" else H, generator=g, device="cuda")


# ---- writing and reading ------------------------------------------------------------------------
def quantized(x, amax):
    """Codes [T, H, D/2] and scales [T, H, D/16] by nvfp4_quantize."""
    T, H, D = x.shape
    rows = x.float().reshape(T * H, D)
    if amax is None:
        r = nv.nvfp4_quantize(rows)
    else:
        r = nv.nvfp4_quantize(rows, gamax_mode="row_given", gamax=amax.expand(H).repeat(T).contiguous())
    return r["codes"].view(T, H, -1), r["scales"].view(T, H, -1)


@pytest.mark.parametrize("T,H,D,P,x,mode", [(1, 1, 64, 16, "bf16", "none"), (37, 3, 128, 64, "bf16", "head"),
                                            (130, 5, 256, 32, "f32", "tensor"), (517, 8, 128, 16, "f32", "head"),
                                            (3001, 2, 64, 128, "bf16", "tensor")])
def test_write_and_read_match_the_quantizer(T, H, D, P, x, mode):
    g = gen(T + D)
    k, v = (normal(g, T, H, D).to(DT[x]) for _ in range(2))
    k[0, 0, :16] = 0.0                                     # a block of zeros
    if T > 30:
        k[7, 0, 3], v[7, 0, 5], v[20, H - 1, 17] = math.inf, math.nan, -math.inf
    ka, va = amaxes(mode, H, g), amaxes(mode, H, g)
    pages = -(-T // P) + 2
    cache = torch.randint(0, 256, (pages, H, P // 16, 18 * D), generator=g, device="cuda", dtype=torch.uint8)
    before = cache.clone()
    slots = torch.randperm(pages * P, generator=g, device="cuda")[:T]
    gone = slots.clone()
    gone[::5] = torch.tensor([-1, pages * P, -(1 << 62), 1 << 62], device="cuda").repeat(T)[:gone[::5].numel()]
    nv.nvfp4_cache_write(cache, k, v, gone, k_gamax=ka, v_gamax=va)
    kept = gone >= 0
    kept &= gone < pages * P
    for part, old, want in zip(parts(cache), parts(before), quantized(k, ka) + quantized(v, va)):
        assert torch.equal(take(part, slots)[kept], want[kept])
        assert torch.equal(take(part, slots)[~kept], take(old, slots)[~kept])
    rest = torch.ones(pages * P, dtype=torch.bool, device="cuda")
    rest[slots[kept]] = False
    other = rest.nonzero().flatten()
    for part, old in zip(parts(cache), parts(before)):
        assert torch.equal(take(part, other), take(old, other))
    for dt in ("bf16", "f32"):
        got = nv.nvfp4_cache_read(cache, gone, k_gamax=ka, v_gamax=va, out_dtype=dt)
        for y, src, a in ((got[0], k, ka), (got[1], v, va)):
            c, s = quantized(src, a)
            mode_kw = {} if a is None else {"gamax_mode": "row_given", "gamax": a.expand(H).repeat(T).contiguous()}
            want = nv.nvfp4_dequantize(c.reshape(T * H, -1), s.reshape(T * H, -1), T * H, D, out_dtype=dt, **mode_kw).view(T, H, D)
            assert torch.equal(y[kept].nan_to_num(), want[kept].nan_to_num())
            assert (y[~kept] == 0).all()


def test_write_takes_slices_of_one_product():
    g = gen(3)
    qkv = normal(g, 50, 12, 128).to(torch.bfloat16)
    slots = torch.arange(50, device="cuda")
    a, b = (nv.nvfp4_cache_empty(4, 16, 4, 128) for _ in range(2))
    nv.nvfp4_cache_write(a, qkv[:, 4:8], qkv[:, 8:], slots)
    nv.nvfp4_cache_write(b, qkv[:, 4:8].contiguous(), qkv[:, 8:].contiguous(), slots)
    assert torch.equal(a, b) and a.any()
    odd = torch.empty(50, 4, 129, device="cuda", dtype=torch.bfloat16)[..., 1:]      # copied: no 16-byte rows
    odd.copy_(qkv[:, 4:8])
    c = nv.nvfp4_cache_empty(4, 16, 4, 128)
    nv.nvfp4_cache_write(c, odd, qkv[:, 8:], slots)
    assert torch.equal(a, c)


# ---- norms and rotation -------------------------------------------------------------------------
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,layout,x,norm", [
    (1, 32, 8, 128, 128, "half", "bf16", True), (1, 1, 1, 16, 16, "half", "f32", True),
    (77, 5, 5, 80, 80, "half", "f32", False), (300, 9, 3, 256, 64, "interleaved", "bf16", True),
    (513, 6, 2, 192, 96, "half", "bf16", True), (40, 4, 4, 512, 512, "interleaved", "f32", True),
    (1200, 8, 1, 64, 32, "interleaved", "f32", False), (9, 3, 1, 48, 0, "half", "bf16", True)])
def test_norm_and_rotation(T, Hq, Hkv, D, rot, layout, x, norm):
    g = gen(T * D)
    qkv = normal(g, T, Hq + 2 * Hkv, D).to(DT[x])
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
    w = [(1 + 0.1 * normal(g, D)).to(DT[x]) for _ in range(2)] if norm else [None, None]
    freq = torch.tensor([1e4 ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float64, device="cuda") if rot else None
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda") if rot else None
    phases = nv.nvfp4_rope_phases(rot, device="cuda") if rot else None
    got = nv.nvfp4_qk_norm_rope(q, k, pos, phases, q_weight=w[0], k_weight=w[1], eps=1e-5, layout=layout, magnitude=1.25)
    for name, t, wt in (("q", q, w[0]), ("k", k, w[1])):
        y = t.double()
        if norm:
            y = y / torch.sqrt(y.square().mean(dim=2, keepdim=True) + 1e-5) * wt.double()
        want = rotate(y, pos, freq, layout, 1.25) if rot else y
        # fp32: the norm about D + 8 roundings, the pair's four products and sums, sin and cos off by 2^-23 and by their
        # angle's error (2^-32 of a turn); then one rounding to x's type
        size = y.abs().amax(dim=2, keepdim=True)
        tol = (D + 24) * 2.0 ** -24 * 1.25 * 2 * size + (2.0 ** -8 if x == "bf16" else 2.0 ** -24) * want.abs()
        assert got[name].dtype == DT[x] and got[name].shape == t.shape
        assert ((got[name].double() - want).abs() <= tol).all()


def test_far_positions_keep_their_angle():
    """Position 2^40 + 5 and a base of 1e4: the turn is a product mod 2^64, compared with whole numbers of Python."""
    phases = nv.nvfp4_rope_phases(64, 10000.0)
    pos = [0, 1, (1 << 40) + 5, (1 << 62) + 12345, -3]
    x = torch.zeros(len(pos), 1, 64, device="cuda")
    x[..., :32] = 1.0                                      # (1, 0) turns to (cos, sin)
    got = nv.nvfp4_qk_norm_rope(x, x, torch.tensor(pos, device="cuda"), phases.cuda())["q"].cpu().double()
    for i, p in enumerate(pos):
        for j in range(32):
            turn = (p * int(phases[j])) % (1 << 64) / 2.0 ** 64
            assert abs(got[i, 0, j].item() - math.cos(2 * math.pi * turn)) < 2.0 ** -22
            assert abs(got[i, 0, 32 + j].item() - math.sin(2 * math.pi * turn)) < 2.0 ** -22


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,layout,x,mode", [
    (1, 8, 2, 128, 128, "half", "bf16", "head"), (133, 6, 3, 64, 32, "half", "f32", "none"),
    (40, 4, 1, 256, 48, "interleaved", "bf16", "tensor"), (2500, 2, 2, 128, 64, "half", "bf16", "none")])
def test_fused_write_is_the_norm_and_rotation_quantized(T, Hq, Hkv, D, rot, layout, x, mode):
    """k goes into the cache as its fp32 value, which fp32 inputs give as an output."""
    g = gen(T + rot)
    qkv = normal(g, T, Hq + 2 * Hkv, D).to(DT[x])
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    w = [(1 + 0.1 * normal(g, D)).to(DT[x]) for _ in range(2)]
    pos = torch.randint(0, 9999, (T,), generator=g, device="cuda")
    ph = nv.nvfp4_rope_phases(rot, device="cuda")
    ka, va = amaxes(mode, Hkv, g), amaxes(mode, Hkv, g)
    pages = -(-T // 32) + 1
    a, b = (nv.nvfp4_cache_empty(pages, 32, Hkv, D) for _ in range(2))
    slots = torch.randperm(pages * 32, generator=g, device="cuda")[:T]
    slots[T // 2] = -1
    r = nv.nvfp4_qk_norm_rope(q, k, pos, ph, q_weight=w[0], k_weight=w[1], layout=layout, cache=a, v=v, slots=slots,
                              k_gamax=ka, v_gamax=va)
    plain = nv.nvfp4_qk_norm_rope(q, k, pos, ph, q_weight=w[0], k_weight=w[1], layout=layout)
    assert set(r) == {"q"} and torch.equal(r["q"], plain["q"])
    wide = nv.nvfp4_qk_norm_rope(q.float(), k.float(), pos, ph, q_weight=w[0], k_weight=w[1], layout=layout)
    nv.nvfp4_cache_write(b, wide["k"], v.float(), slots, k_gamax=ka, v_gamax=va)
    assert torch.equal(a, b)


# ---- attention ----------------------------------------------------------------------------------
class Paged:
    """Sequences of the given lengths in a cache whose other bytes are NaN scales and garbage."""

    def __init__(self, seed, lens, H, D, P, mode="none", spare=3, scale=1.0):
        g = gen(seed)
        self.lens, self.H, self.D, self.P = lens, H, D, P
        need = [-(-n // P) for n in lens]
        total = sum(need) + spare
        self.cache = torch.full((total, H, P // 16, 18 * D), 255, dtype=torch.uint8, device="cuda")
        order = torch.randperm(total, generator=g, device="cuda")
        self.pages = torch.full((len(lens), max(max(need), 1)), -7, dtype=torch.int32, device="cuda")
        self.ka, self.va = amaxes(mode, H, g), amaxes(mode, H, g)
        at = 0
        for b, (n, p) in enumerate(zip(lens, need)):
            self.pages[b, :p] = order[at:at + p].int()
            at += p
            if n:
                k, v = normal(g, n, H, D) * scale, normal(g, n, H, D)
                nv.nvfp4_cache_write(self.cache, k, v, self.slots(b), k_gamax=self.ka, v_gamax=self.va)
        self.lengths = torch.tensor(lens, device="cuda")

    def slots(self, b):
        j = torch.arange(self.lens[b], device="cuda")
        return self.pages[b].long()[j // self.P] * self.P + j % self.P

    def values(self, b):
        kc, ks, vc, vs = (take(p, self.slots(b)) for p in parts(self.cache))
        return values(kc, ks, self.ka), values(vc, vs, self.va)

    def check(self, q, counts, got, lse=None, **kw):
        D = self.D
        kw.setdefault("scale", D ** -0.5)
        row = 0
        for b, n in enumerate(counts):
            if n == 0:
                continue
            k, v = self.values(b)
            out, want, mass, most = attention(q[row:row + n], k, v, n, **kw)
            biggest = v.abs().max().item() if v.numel() else 0.0
            tol = tolerance(out, mass, most, biggest, self.lens[b], D, q.dtype, got.dtype)
            off = (got[row:row + n].double() - out).abs()
            assert (off <= tol).all(), (b, (off / tol).max().item())
            if lse is not None:
                inf = torch.isneginf(want)
                assert torch.equal(torch.isneginf(lse[row:row + n]), inf)
                d = (lse[row:row + n].double() - want).abs()[~inf]
                assert (d <= (D + 8) * 2.0 ** -23 * most + 2.0 ** -22 * want.abs()[~inf] + (self.lens[b] / 16 + 64) * 2.0 ** -23).all()
            row += n


CASES = [
    # lens, n (None: one each, no offsets), Hq, H, D, P, x, mode, options
    ([1], None, 1, 1, 64, 16, "bf16", "none", {}),
    ([200], None, 32, 8, 128, 64, "bf16", "head", {}),
    ([15, 16, 17, 31, 0, 513], None, 8, 8, 128, 16, "bf16", "tensor", {}),
    ([40000], None, 16, 2, 128, 64, "bf16", "head", {}),
    ([5000, 3, 12000, 0, 77], None, 5, 1, 64, 128, "bf16", "none", {"sinks": True}),
    ([700, 9000, 1], None, 16, 4, 256, 32, "bf16", "tensor", {"causal": False}),
    ([3000, 257], None, 24, 2, 128, 32, "f32", "head", {}),
    ([900, 2000, 33], [3, 1, 5], 15, 3, 64, 16, "f32", "tensor", {"window": 100, "sinks": True}),
    ([64, 2, 600, 5], [4, 7, 0, 5], 8, 2, 128, 16, "bf16", "none", {}),
    ([64, 2, 600, 5], [4, 7, 0, 5], 8, 2, 128, 16, "f32", "none", {"causal": False, "window": 3}),
    ([1500, 100], [200, 100], 6, 2, 128, 64, "bf16", "head", {}),
    ([1500, 100], [200, 100], 6, 2, 64, 64, "bf16", "head", {"window": 77}),
    ([2100], [300], 4, 4, 256, 64, "bf16", "none", {}),
    ([2100], [70], 4, 4, 256, 64, "f32", "none", {"window": 1}),
    ([0, 0], None, 4, 2, 128, 16, "bf16", "none", {}),
    ([0, 0], None, 4, 2, 128, 16, "f32", "none", {"sinks": True}),
    ([700 + 13 * i for i in range(70)], None, 16, 2, 128, 16, "bf16", "head", {}),
    ([1 + i % 40 for i in range(100)], None, 3, 3, 64, 16, "bf16", "none", {}),
    # many rows a sequence (the tensor-memory kernel), next to few, none, and queries before the first key
    ([64], [64], 2, 1, 128, 16, "bf16", "none", {}),
    ([65], [65], 1, 1, 64, 16, "bf16", "head", {}),
    ([1000, 5, 0, 129, 3000], [300, 5, 0, 129, 1], 8, 2, 128, 32, "bf16", "head", {"sinks": True}),
    ([1000, 5, 0, 129, 3000], [300, 5, 0, 129, 1], 8, 2, 64, 16, "bf16", "tensor", {"window": 200}),
    ([40, 513, 0], [100, 70, 80], 5, 1, 128, 48, "bf16", "none", {}),
    ([700, 900], [700, 900], 6, 2, 128, 64, "bf16", "none", {"causal": False, "window": 64}),
    ([5000], [257], 4, 4, 128, 64, "bf16", "tensor", {}),
    ([400 + 37 * i for i in range(30)], [65 + 7 * i for i in range(30)], 6, 3, 64, 16, "bf16", "none", {}),
    ([900], [450], 12, 4, 128, 64, "bf16", "head", {"window": 1}),
    ([900], [450], 12, 4, 128, 64, "bf16", "head", {"scale": -0.05}),
    # many heads a KV head without offsets; sequences on both sides of what the tensor-memory kernel takes
    ([9000, 300, 5000], None, 80, 1, 128, 64, "bf16", "head", {}),
    ([5461, 5462, 2000, 4096, 4095], [6, 6, 17, 8, 8], 8, 1, 128, 32, "bf16", "none", {"causal": False}),
    ([5461, 5462, 2000, 4096, 4095], [6, 6, 17, 8, 8], 8, 1, 64, 32, "bf16", "tensor", {"sinks": True, "window": 3000}),
    ([3000, 2500], [300, 257], 8, 2, 128, 64, "bf16", "none", {"window": 1000}),
    ([300, 600, 513, 0, 1], [1000, 900, 700, 80, 700], 5, 1, 128, 48, "bf16", "none", {}),
    ([300, 600, 513, 0, 1], [1000, 900, 700, 80, 700], 5, 1, 64, 48, "bf16", "head", {"sinks": True, "window": 20}),
    ([1100 + 37 * i for i in range(30)], [129 + 7 * i for i in range(30)], 6, 3, 64, 16, "bf16", "none", {}),
    ([2048, 4096], [2048, 130], 4, 2, 64, 64, "bf16", "none", {}),
    ([1024, 1023, 1], None, 24, 1, 128, 64, "bf16", "none", {}),
    ([1100, 30, 0], None, 256, 1, 64, 16, "bf16", "head", {}),
    ([30000, 5, 470], None, 8, 2, 128, 64, "bf16", "head", {"window": 500}),
    ([30000, 5, 470], [3, 5, 2], 8, 2, 64, 64, "f32", "head", {"window": 1100, "sinks": True}),
    ([1500, 1025, 1], None, 24, 1, 64, 64, "bf16", "none", {"sinks": True}),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_attention(i):
    lens, counts, Hq, H, D, P, x, mode, opt = CASES[i]
    opt = dict(opt)
    c = Paged(i, lens, H, D, P, mode)
    g = gen(100 + i)
    n = [1] * len(lens) if counts is None else counts
    q = (2.0 * normal(g, sum(n), Hq, D)).to(DT[x])
    if opt.get("sinks"):
        opt["sinks"] = normal(g, Hq)
    off = None if counts is None else torch.tensor([0] + counts, device="cuda").cumsum(0)
    for o in ("bf16", "f32") if x == "bf16" else ("f32",):
        got, lse = nv.nvfp4_cache_attention(q, c.cache, c.pages, c.lengths, offsets=off, k_gamax=c.ka, v_gamax=c.va,
                                            out_dtype=o, want_lse=True, **opt)
        c.check(q, n, got, lse, **opt)
        again = nv.nvfp4_cache_attention(q, c.cache, c.pages, c.lengths, offsets=off, k_gamax=c.ka, v_gamax=c.va,
                                         out_dtype=o, **opt)
        assert torch.equal(got, again)
